// The selective state space scan, its gradient and its single-token step.
//
//   dt = softplus(raw + bias) or raw,   a_t = e^(A dt_t)
//   h_t = a_t h_{t-1} + dt_t x_t B_t^T,   y_t = h_t C_t + D x_t
//
// per head, with a state h of P x S.  One token after the other this is
// 4 P S flop a token and head that no matrix instruction takes.  Over a chunk
// of Q tokens with the sums  c_i = sum_{j<=i} A dt_j  it is products of
// matrices (i, j tokens of the chunk, h_0 the state it starts from):
//
//   y_i   = sum_{j<=i} M_ij x_j + e^{c_i} h_0 C_i + D x_i,  M_ij = (C_i . B_j) e^{c_i - c_j} dt_j
//   h_Q   = e^{c_Q} h_0 + sum_j e^{c_Q - c_j} dt_j x_j B_j^T
//
// All exponents are differences of the sums, at most 0 for A < 0, so nothing
// overflows however long the chunk is.  With u the gradient of h_Q and dy that
// of y (dP_ij = dy_i . x_j):
//
//   dxdt_j = sum_{i>=j} (M_ij / dt_j) dy_i + e^{c_Q - c_j} u B_j
//   dC_i   = sum_j dS_ij B_j + e^{c_i} dy_i h_0,            dS_ij = dP_ij e^{c_i - c_j} dt_j  (i >= j)
//   dB_j   = sum_i dS_ij C_i + e^{c_Q - c_j} dt_j x_j u
//   dh_0   = e^{c_Q} u + sum_i e^{c_i} dy_i C_i^T
//   dl_t   = sum_{j<t<=i} W_ij + sum_{i>=t} e^{c_i} (dy_i h_0) . C_i
//          + sum_{j<t} dt_j e^{c_Q - c_j} (u B_j) . x_j + e^{c_Q} <h_0, u>,   W_ij = dS_ij (C_i . B_j)
//
// (dl_t the gradient of A dt_t: every path that crosses the decay of step t).
//
// Numbers.  The matrix instructions take bf16 operands and add in fp32.  x, B,
// C and dy are bf16 already; what is computed on the way (M, the states, dS)
// enters as the sum of two or three bf16 numbers, each the rounding of what
// the ones before it left, so that 16 or 24 bits of it take part.  fp32 calls
// run on the fp32 matrix instructions instead.  States, sums and exponents are
// fp32, the running sums c_i are added in fp64.
//
// Fragments (16x16 blocks, 64 lanes, q = lane / 16): an operand's lane holds 8
// values of the reduction for row (or column) lane % 16, a result's lane four
// rows 4q..4q+3 of column lane % 16.  The order of the reduction is free as
// long as both operands agree, so two results of 16 rows are an operand of a
// reduction over 32 as they stand: states never leave the registers.  Operands
// whose reduction runs down the columns of a tile come from LDS through the
// transposing read.
#pragma once

#include "seq_common.h"

namespace convfwd {

struct ScanParams {
    const void *x, *dt, *b, *c;
    const float *a, *d, *dt_bias, *state;
    const int32_t *lengths;
    void *y;
    float *state_out;
    int64_t x_ld, dt_ld, b_ld, c_ld, y_ld;
    int64_t L;
    int N, H, P, G, S, NPB;     // NPB: blocks of 64 channels of a head
    int K;                      // chunks of a sequence
    int nseg, seg;              // segments of a sequence, chunks of a segment
    int softplus, vec;
    float *seg_state, *seg_log; // [unit][nseg][SP][64], [unit][nseg]
    float *bound;               // [unit][K][SP][64]: the state (or its gradient) at every chunk's border
    // gradient
    const void *dy;
    const float *dstate_out;
    void *dx, *ddt, *db, *dc;
    float *dstate;
    int64_t dy_ld, dx_ld, ddt_ld, db_ld, dc_ld;
    const float *ubound;        // as bound, of the gradient
    float *part_head;           // [3][N * K][H]: dA, ddt_bias, dD
    float *part_b, *part_c;     // [slices][N * L][G][SP]
    int slices, heads_per_slice;
};

constexpr int kPB = 64;         // channels of a head that one workgroup takes

// ---- fragments ---------------------------------------------------------------
template <typename T> struct Frag;
template <> struct Frag<bf16_t> {
    static constexpr int Q = 64;            // tokens of a chunk
    static constexpr int VE = 8;            // elements of 16 bytes
    static constexpr int PAD = 8;           // row padding of the LDS tiles, elements: 16 bytes
    typedef bf16x8 type;
};
template <> struct Frag<float> {
    static constexpr int Q = 32;
    static constexpr int VE = 4;
    static constexpr int PAD = 4;
    struct type { float v[8]; };
};

SEQ_DEV f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
SEQ_DEV f32x4 mma(const Frag<float>::type &a, const Frag<float>::type &b, f32x4 c)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
}

// v as the sum of NS bf16 fragments (or itself in fp32)
template <typename T, int NS> struct Split {
    typename Frag<T>::type f[NS];
};
template <int NS> SEQ_DEV void make_split(const float (&v)[8], Split<bf16_t, NS> &s)
{
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s.f[k][e] = (bf16_t)r[e];
            r[e] -= (float)s.f[k][e];
        }
}
template <int NS> SEQ_DEV void make_split(const float (&v)[8], Split<float, NS> &s)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) s.f[0].v[e] = v[e];
}
// fp32 needs one term only
template <typename T, int NS> constexpr int terms() { return sizeof(T) == 4 ? 1 : NS; }

template <typename T, int NS> SEQ_DEV f32x4 mma_a(const Split<T, NS> &a, const typename Frag<T>::type &b, f32x4 c)
{
#pragma unroll
    for (int k = 0; k < NS; ++k) c = mma(a.f[k], b, c);
    return c;
}
template <typename T, int NS> SEQ_DEV f32x4 mma_b(const typename Frag<T>::type &a, const Split<T, NS> &b, f32x4 c)
{
#pragma unroll
    for (int k = 0; k < NS; ++k) c = mma(a, b.f[k], c);
    return c;
}

SEQ_DEV float frag_get(bf16x8 f, int e) { return (float)f[e]; }
SEQ_DEV float frag_get(const Frag<float>::type &f, int e) { return f.v[e]; }

// Row row0 + lane % 16 of an LDS tile, reduction indices k0 + 8q .. k0 + 8q + 7
SEQ_DEV bf16x8 read_rows(const bf16_t *t, int ld, int row0, int k0, int lane)
{
    return *reinterpret_cast<const bf16x8 *>(t + (row0 + (lane & 15)) * ld + k0 + (lane >> 4) * 8);
}
SEQ_DEV Frag<float>::type read_rows(const float *t, int ld, int row0, int k0, int lane)
{
    const f32x4 *p = reinterpret_cast<const f32x4 *>(t + (row0 + (lane & 15)) * ld + k0 + (lane >> 4) * 8);
    const f32x4 a = p[0], b = p[1];
    Frag<float>::type f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = a[e], f.v[4 + e] = b[e];
    return f;
}

// The same row, in the order in which two results stacked over 32 rows hold
// them: k0 + 4q .. +3, then k0 + 16 + 4q .. +3
SEQ_DEV bf16x8 read_rows_stacked(const bf16_t *t, int ld, int row0, int k0, int lane)
{
    const bf16_t *p = t + (row0 + (lane & 15)) * ld + k0 + (lane >> 4) * 4;
    const bf16x4 a = *reinterpret_cast<const bf16x4 *>(p), b = *reinterpret_cast<const bf16x4 *>(p + 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
SEQ_DEV Frag<float>::type read_rows_stacked(const float *t, int ld, int row0, int k0, int lane)
{
    const float *p = t + (row0 + (lane & 15)) * ld + k0 + (lane >> 4) * 4;
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 16);
    Frag<float>::type f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = a[e], f.v[4 + e] = b[e];
    return f;
}

// Column col0 + lane % 16, reduction over the tile's rows k0 + 8q .. k0 + 8q + 7.
// The transposing read takes 4 rows of 16 columns with each 16 lanes (lane i
// points at row i / 4, columns 4 (i % 4) ..) and leaves lane i with column i.
SEQ_DEV bf16x8 read_cols(const bf16_t *t, int ld, int k0, int col0, int lane)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
    const bf16_t *p = t + (k0 + (lane >> 4) * 8 + ((lane & 15) >> 2)) * ld + col0 + (lane & 3) * 4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * ld));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
}
SEQ_DEV Frag<float>::type read_cols(const float *t, int ld, int k0, int col0, int lane)
{
    const float *p = t + (k0 + (lane >> 4) * 8) * ld + col0 + (lane & 15);
    Frag<float>::type f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = p[e * ld];
    return f;
}

// four consecutive elements of an LDS row, as the k-th term of a split
template <int NS, typename T> SEQ_DEV void write_split4(T *t, int term_stride, f32x4 v)
{
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4 *>(t) = v;
    } else {
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            bf16x4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[e] = (bf16_t)v[e];
                v[e] -= (float)h[e];
            }
            *reinterpret_cast<bf16x4 *>(t + k * term_stride) = h;
        }
    }
}

// ---- tiles -------------------------------------------------------------------
// ROWS x COLS of a matrix with `ld` elements from row to row, through 256
// threads' registers into LDS; zeros outside `rows` x `cols`, which are never
// read (they may hold anything).
template <typename T, int ROWS, int COLS> struct Tile {
    static constexpr int VE = Frag<T>::VE;
    static constexpr int NV = ROWS * COLS / VE / 256;
    static constexpr int LD = COLS + Frag<T>::PAD;
    static constexpr int CV = COLS / VE;
    static_assert(ROWS * COLS % (VE * 256) == 0, "whole vectors per thread");
    typedef typename Pack<T, VE>::type vec_t;
    vec_t v[NV];

    SEQ_DEV void load(const T *g, int64_t ld, int rows, int cols, bool vec)
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = threadIdx.x + k * 256, r = e / CV, c = (e - r * CV) * VE;
            vec_t q = {};
            if (r < rows && c < cols) {
                const T *p = g + r * ld + c;
                if (vec) {
                    q = *reinterpret_cast<const vec_t *>(p);
                } else {
#pragma unroll
                    for (int i = 0; i < VE; ++i)
                        if (c + i < cols) q[i] = p[i];
                }
            }
            v[k] = q;
        }
    }
    SEQ_DEV void store(T *lds) const
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = threadIdx.x + k * 256, r = e / CV, c = (e - r * CV) * VE;
            *reinterpret_cast<vec_t *>(lds + r * LD + c) = v[k];
        }
    }
    // the inverse way, from LDS to memory
    static SEQ_DEV void write(const T *lds, T *g, int64_t ld, int rows, int cols, bool vec)
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = threadIdx.x + k * 256, r = e / CV, c = (e - r * CV) * VE;
            if (r >= rows || c >= cols) continue;
            const vec_t q = *reinterpret_cast<const vec_t *>(lds + r * LD + c);
            T *p = g + r * ld + c;
            if (vec) {
                *reinterpret_cast<vec_t *>(p) = q;
            } else {
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    if (c + i < cols) p[i] = q[i];
            }
        }
    }
    static SEQ_DEV void write_zeros(T *g, int64_t ld, int rows, int cols, bool vec)
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = threadIdx.x + k * 256, r = e / CV, c = (e - r * CV) * VE;
            if (r >= rows || c >= cols) continue;
            T *p = g + r * ld + c;
            if (vec) {
                *reinterpret_cast<vec_t *>(p) = vec_t{};
            } else {
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    if (c + i < cols) p[i] = (T)0.0f;
            }
        }
    }
};

// ---- wave helpers --------------------------------------------------------------
// inclusive sums over the 64 lanes
SEQ_DEV double wave_prefix(double v, int lane)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}
SEQ_DEV float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
// the sum over the 16 lanes of a row, in every one of them
SEQ_DEV float row_sum(float v)
{
#define SEQ_ROR(n) \
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + n, 0xf, 0xf, true))
    SEQ_ROR(8);
    SEQ_ROR(4);
    SEQ_ROR(2);
    SEQ_ROR(1);
#undef SEQ_ROR
    return v;
}

// Token `lane` of a chunk: the step size dt (0 behind the sequence) and the
// running sum of log2 of the decays.  The products and the sum are in fp64:
// the exponents used later are differences of these sums.
SEQ_DEV void chunk_decay(float raw, bool live, float a, int softplus_on, int lane, float &dt, float &cum)
{
    dt = live ? (softplus_on ? softplus(raw) : raw) : 0.0f;
    cum = (float)wave_prefix((double)a * (double)dt * 1.4426950408889634074, lane);
}

SEQ_DEV float wave_last(float v) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63)); }

// ---- states at the chunks' borders, and at the segments' ------------------------
// One workgroup: 64 channels of a head, one segment of chunks, wave w the
// channels 16w..16w+15 and all of the state (results: rows channels, columns
// states).  REV runs from the last chunk to the first with dy, C and weights
// e^{c_i} instead of x, B and e^{c_Q - c_j} dt_j: the state's gradient.  STORE
// leaves the state at every chunk's near border in `bound` and starts from the
// segment's own start; without it the segment starts from zero and leaves its
// last state and the logarithm of its decay.
template <typename T, int SP, bool REV, bool STORE>
__global__ void __launch_bounds__(256) scan_state_kernel(ScanParams p)
{
    constexpr int Q = Frag<T>::Q, NT = SP / 16, NS = terms<T, 3>();
    typedef Tile<T, Q, kPB> XT;
    typedef Tile<T, Q, SP> BT;
    __shared__ __align__(16) T sX[Q * XT::LD];
    __shared__ __align__(16) T sB[Q * BT::LD];
    __shared__ float sW[Q], sTot[1];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane >> 4;
    const int nseg = STORE ? p.nseg : p.nseg - 1;
    const int64_t unit = blockIdx.x / nseg;
    const int s0 = (int)(blockIdx.x - unit * nseg);
    const int seg = STORE ? s0 : REV ? s0 + 1 : s0;      // the last segment of the run is not needed
    const int pb = (int)(unit % p.NPB);
    const int64_t nh = unit / p.NPB, n = nh / p.H;
    const int h = (int)(nh - n * p.H), g = h / (p.H / p.G);
    const int64_t len = seq_len(p.lengths, n, p.L);
    const int pcols = min(kPB, p.P - pb * kPB);
    const T *xg = (const T *)(REV ? p.dy : p.x) + n * p.L * (REV ? p.dy_ld : p.x_ld) + (int64_t)h * p.P + pb * kPB;
    const T *bg = (const T *)(REV ? p.c : p.b) + n * p.L * (REV ? p.c_ld : p.b_ld) + (int64_t)g * p.S;
    const T *dg = (const T *)p.dt + n * p.L * p.dt_ld + h;
    const int64_t x_ld = REV ? p.dy_ld : p.x_ld, b_ld = REV ? p.c_ld : p.b_ld;
    const float a = p.a[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
    const int c_lo = seg * p.seg, c_hi = min(p.K, c_lo + p.seg);
    const int c_live = (int)min((int64_t)c_hi, (len + Q - 1) / Q);   // chunks behind the sequence change nothing
    const bool busy = w * 16 < pcols;

    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    const int ch = w * 16 + q * 4;      // the first of this lane's four channels
    if (STORE) {
        if (p.nseg > 1) {
            const float *s = p.seg_state + (unit * p.nseg + seg) * (SP * kPB);
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = *reinterpret_cast<const f32x4 *>(s + (t * 16 + (lane & 15)) * kPB + ch);
        } else {
            const float *s = REV ? p.dstate_out : p.state;
            if (s) {
                s += (nh * p.P + pb * kPB) * p.S;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (ch + r < pcols && t * 16 + (lane & 15) < p.S)
                            acc[t][r] = s[(int64_t)(ch + r) * p.S + t * 16 + (lane & 15)];
            }
        }
    }

    XT xt;
    BT bt;
    float raw = 0.0f, log_dec = 0.0f;
    auto fetch = [&](int c) __attribute__((always_inline)) {
        const int64_t t0 = (int64_t)c * Q;
        const int rows = (int)min((int64_t)Q, len - t0);
        xt.load(xg + t0 * x_ld, x_ld, rows, pcols, p.vec);
        bt.load(bg + t0 * b_ld, b_ld, rows, p.S, p.vec);
        if (w == 0) raw = lane < rows ? (float)dg[(t0 + lane) * p.dt_ld] + bias : 0.0f;
    };
    if (c_lo < c_live) fetch(REV ? c_live - 1 : c_lo);
    for (int k = c_lo; k < c_live; ++k) {
        const int c = REV ? c_live - 1 - (k - c_lo) : k;
        __syncthreads();
        xt.store(sX);
        bt.store(sB);
        if (w == 0) {
            float dt, cum;
            chunk_decay(raw, (int64_t)c * Q + lane < len && lane < Q, a, p.softplus, lane, dt, cum);
            const float tot = wave_last(cum);
            if (lane < Q) sW[lane] = REV ? exp2_fast(cum) : exp2_fast(tot - cum) * dt;
            if (lane == 0) sTot[0] = tot;
        }
        __syncthreads();
        if (k + 1 < c_live) fetch(REV ? c - 1 : c + 1);
        if (STORE) {
            float *s = p.bound + (unit * p.K + c) * (SP * kPB);
#pragma unroll
            for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4 *>(s + (t * 16 + (lane & 15)) * kPB + ch) = acc[t];
        }
        const float tot = sTot[0], dec = exp2_fast(tot);
        log_dec += tot;
        if (busy) {
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] *= dec;
#pragma unroll
            for (int ks = 0; ks < Q / 32; ++ks) {
                const typename Frag<T>::type xf = read_cols(sX, XT::LD, ks * 32, w * 16, lane);
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = frag_get(xf, e) * sW[ks * 32 + q * 8 + e];
                Split<T, NS> xs;
                make_split(v, xs);
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t] = mma_a(xs, read_cols(sB, BT::LD, ks * 32, t * 16, lane), acc[t]);
            }
        }
    }
    if (!STORE) {
        float *s = p.seg_state + (unit * p.nseg + seg) * (SP * kPB);
#pragma unroll
        for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4 *>(s + (t * 16 + (lane & 15)) * kPB + ch) = acc[t];
        if (threadIdx.x == 0) p.seg_log[unit * p.nseg + seg] = log_dec;
    } else if (REV && seg == 0 && p.dstate) {
        float *s = p.dstate + (nh * p.P + pb * kPB) * p.S;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (ch + r < pcols && t * 16 + (lane & 15) < p.S)
                    s[(int64_t)(ch + r) * p.S + t * 16 + (lane & 15)] = acc[t][r];
    }
}

// Joins the segments: what each left from zero becomes the state it starts
// from, one thread per element of the state, segments in order.
template <int SP, bool REV> __global__ void __launch_bounds__(256) scan_join_kernel(ScanParams p)
{
    constexpr int BLK = SP * kPB / 256;
    const int64_t unit = blockIdx.x / BLK;
    const int e = (int)(blockIdx.x - unit * BLK) * 256 + threadIdx.x;
    const int pb = (int)(unit % p.NPB), s = e / kPB, ch = pb * kPB + (e & (kPB - 1));
    const int64_t nh = unit / p.NPB;
    const float *first = REV ? p.dstate_out : p.state;
    float cur = first && s < p.S && ch < p.P ? first[(nh * p.P + ch) * p.S + s] : 0.0f;
    float *v = p.seg_state + unit * p.nseg * (SP * kPB) + e;
    const float *lg = p.seg_log + unit * p.nseg;
    for (int k = 0; k < p.nseg; ++k) {
        const int seg = REV ? p.nseg - 1 - k : k;
        const bool last = k == p.nseg - 1;
        const float add = last ? 0.0f : v[(int64_t)seg * (SP * kPB)];
        const float dec = last ? 0.0f : exp2_fast(lg[seg]);
        v[(int64_t)seg * (SP * kPB)] = cur;
        cur = fmaf(dec, cur, add);
    }
}

// Lower-triangle tile t of the chunk's scores: row it, column jt <= it
SEQ_DEV void tri_tile(int t, int &it, int &jt)
{
    it = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
    jt = t - it * (it + 1) / 2;
}

// ---- forward -------------------------------------------------------------------
// One workgroup: 64 channels of a head, one segment of chunks; wave w keeps the
// state of channels 16w..16w+15 in registers (results: rows states, columns
// channels, which makes them the operand of h_0 C as they stand).  The chunk's
// scores are computed once, their 16x16 tiles dealt to the waves, and pass
// through LDS as M.
template <typename T, int SP> __global__ void __launch_bounds__(256, 2) scan_fwd_kernel(ScanParams p)
{
    constexpr int Q = Frag<T>::Q, NT = SP / 16, NI = Q / 16, TRI = NI * (NI + 1) / 2, TPW = (TRI + 3) / 4;
    constexpr int NM = terms<T, 2>(), NX = terms<T, 3>(), MLD = Q + Frag<T>::PAD;
    typedef Tile<T, Q, kPB> XT;
    typedef Tile<T, Q, SP> BT;
    __shared__ __align__(16) T sX[Q * XT::LD];
    __shared__ __align__(16) T sB[Q * BT::LD];
    __shared__ __align__(16) T sC[Q * BT::LD];
    __shared__ __align__(16) T sM[NM * Q * MLD];
    __shared__ __align__(16) float sCum[Q], sDt[Q];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane >> 4;
    const int64_t unit = blockIdx.x / p.nseg;
    const int seg = (int)(blockIdx.x - unit * p.nseg);
    const int pb = (int)(unit % p.NPB);
    const int64_t nh = unit / p.NPB, n = nh / p.H;
    const int h = (int)(nh - n * p.H), g = h / (p.H / p.G);
    const int64_t len = seq_len(p.lengths, n, p.L);
    const int pcols = min(kPB, p.P - pb * kPB);
    const T *xg = (const T *)p.x + n * p.L * p.x_ld + (int64_t)h * p.P + pb * kPB;
    const T *bg = (const T *)p.b + n * p.L * p.b_ld + (int64_t)g * p.S;
    const T *cg = (const T *)p.c + n * p.L * p.c_ld + (int64_t)g * p.S;
    const T *dg = (const T *)p.dt + n * p.L * p.dt_ld + h;
    T *yg = (T *)p.y + n * p.L * p.y_ld + (int64_t)h * p.P + pb * kPB;
    const float a = p.a[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f, skip = p.d ? p.d[h] : 0.0f;
    const int c_lo = seg * p.seg, c_hi = min(p.K, c_lo + p.seg);
    const int c_live = (int)min((int64_t)c_hi, (len + Q - 1) / Q);
    const bool busy = w * 16 < pcols;
    const int col = w * 16 + (lane & 15);       // this lane's channel

    f32x4 st[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) st[t] = f32x4{0, 0, 0, 0};
    if (p.nseg > 1) {
        const float *s = p.seg_state + (unit * p.nseg + seg) * (SP * kPB) + col;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) st[t][r] = s[(t * 16 + q * 4 + r) * kPB];
    } else if (p.state && col < pcols) {
        const float *s = p.state + (nh * p.P + pb * kPB + col) * p.S;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (t * 16 + q * 4 + r < p.S) st[t][r] = s[t * 16 + q * 4 + r];
    }
    // the tiles of M above the diagonal that a reduction over 32 tokens meets
    for (int e = threadIdx.x; e < NM * Q * MLD; e += 256) sM[e] = (T)0.0f;

    XT xt;
    BT bt, ct;
    float raw = 0.0f;
    auto fetch = [&](int c) __attribute__((always_inline)) {
        const int64_t t0 = (int64_t)c * Q;
        const int rows = (int)min((int64_t)Q, len - t0);
        xt.load(xg + t0 * p.x_ld, p.x_ld, rows, pcols, p.vec);
        bt.load(bg + t0 * p.b_ld, p.b_ld, rows, p.S, p.vec);
        ct.load(cg + t0 * p.c_ld, p.c_ld, rows, p.S, p.vec);
        if (w == 0) raw = lane < rows ? (float)dg[(t0 + lane) * p.dt_ld] + bias : 0.0f;
    };
    if (c_lo < c_live) fetch(c_lo);
    for (int c = c_lo; c < c_live; ++c) {
        const int64_t t0 = (int64_t)c * Q;
        __syncthreads();
        xt.store(sX);
        bt.store(sB);
        ct.store(sC);
        if (w == 0) {
            float dt, cum;
            chunk_decay(raw, t0 + lane < len && lane < Q, a, p.softplus, lane, dt, cum);
            if (lane < Q) {
                sDt[lane] = dt;
                sCum[lane] = cum;
            }
        }
        __syncthreads();
        if (c + 1 < c_live) fetch(c + 1);
        // M, tile by tile: rows j, column i in a lane, so four neighbours of a row of M
#pragma unroll
        for (int k = 0; k < TPW; ++k) {
            const int t = w + 4 * k;
            if (t < TRI) {
                int it, jt;
                tri_tile(t, it, jt);
                f32x4 s = {0, 0, 0, 0};
#pragma unroll
                for (int ks = 0; ks < SP / 32; ++ks)
                    s = mma(read_rows(sB, BT::LD, jt * 16, ks * 32, lane), read_rows(sC, BT::LD, it * 16, ks * 32, lane), s);
                const int i = it * 16 + (lane & 15), j = jt * 16 + q * 4;
                const float ci = sCum[i];
                const f32x4 cj = *reinterpret_cast<const f32x4 *>(sCum + j), dj = *reinterpret_cast<const f32x4 *>(sDt + j);
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] = i >= j + r ? s[r] * exp2_fast(ci - cj[r]) * dj[r] : 0.0f;
                write_split4<NM>(sM + i * MLD + j, Q * MLD, s);
            }
        }
        __syncthreads();
        if (busy) {
            f32x4 y[NI];
#pragma unroll
            for (int it = 0; it < NI; ++it) y[it] = f32x4{0, 0, 0, 0};
            // e^{c_i} h_0 C_i
#pragma unroll
            for (int ks = 0; ks < SP / 32; ++ks) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = st[2 * ks][e], v[4 + e] = st[2 * ks + 1][e];
                Split<T, NM> hs;
                make_split(v, hs);
#pragma unroll
                for (int it = 0; it < NI; ++it)
                    y[it] = mma_b(read_rows_stacked(sC, BT::LD, it * 16, ks * 32, lane), hs, y[it]);
            }
#pragma unroll
            for (int it = 0; it < NI; ++it) {
                const f32x4 ci = *reinterpret_cast<const f32x4 *>(sCum + it * 16 + q * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) y[it][r] *= exp2_fast(ci[r]);
            }
            const float tot = sCum[Q - 1], dec = exp2_fast(tot);
#pragma unroll
            for (int t = 0; t < NT; ++t) st[t] *= dec;
#pragma unroll
            for (int ks = 0; ks < Q / 32; ++ks) {
                const typename Frag<T>::type xf = read_cols(sX, XT::LD, ks * 32, w * 16, lane);
#pragma unroll
                for (int it = 2 * ks; it < NI; ++it)
#pragma unroll
                    for (int m = 0; m < NM; ++m)
                        y[it] = mma(read_rows(sM + m * Q * MLD, MLD, it * 16, ks * 32, lane), xf, y[it]);
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = ks * 32 + q * 8 + e;
                    v[e] = frag_get(xf, e) * (exp2_fast(tot - sCum[j]) * sDt[j]);
                }
                Split<T, NX> xs;
                make_split(v, xs);
#pragma unroll
                for (int t = 0; t < NT; ++t) st[t] = mma_b(read_cols(sB, BT::LD, ks * 32, t * 16, lane), xs, st[t]);
            }
            // y in place of this wave's own columns of x
#pragma unroll
            for (int it = 0; it < NI; ++it)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    T *o = sX + (it * 16 + q * 4 + r) * XT::LD + col;
                    *o = (T)fmaf(skip, (float)*o, y[it][r]);
                }
        }
        __syncthreads();
        // rows behind the sequence come out as zeros: x and C are zeros there
        XT::write(sX, yg + t0 * p.y_ld, p.y_ld, (int)min((int64_t)Q, p.L - t0), pcols, p.vec);
    }
    for (int c = max(c_lo, c_live); c < c_hi; ++c) {
        const int64_t t0 = (int64_t)c * Q;
        XT::write_zeros(yg + t0 * p.y_ld, p.y_ld, (int)min((int64_t)Q, p.L - t0), pcols, p.vec);
    }
    if (p.state_out && seg == p.nseg - 1 && col < pcols) {
        float *s = p.state_out + (nh * p.P + pb * kPB + col) * p.S;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (t * 16 + q * 4 + r < p.S) s[t * 16 + q * 4 + r] = st[t][r];
    }
}

// ---- gradient ------------------------------------------------------------------
// One workgroup: one chunk of one group, a slice of the group's heads one after
// the other.  C . B is the same for all of them and stays in registers, and so
// do the sums of dS over the heads, from which dB and dC get their parts inside
// the chunk by one product each at the end.  The waves share dP's 16x16 tiles
// as the forward shares its scores; dx goes by channels (wave w: 16w..), dB and
// dC by states (wave w: the 16-state tiles w, w + 4).  The states at the chunk's
// borders and their gradients come from memory, where the two runs of
// scan_state_kernel left them.
template <typename T, int SP> __global__ void __launch_bounds__(256) scan_bwd_kernel(ScanParams p)
{
    constexpr int Q = Frag<T>::Q, NT = SP / 16, NI = Q / 16, TRI = NI * (NI + 1) / 2, TPW = (TRI + 3) / 4;
    constexpr int NS = terms<T, 3>(), MLD = Q + Frag<T>::PAD, NTW = (NT + 3) / 4, ULD = kPB + Frag<T>::PAD;
    typedef Tile<T, Q, kPB> XT;
    typedef Tile<T, Q, SP> BT;
    typedef typename Frag<T>::type frag;
    __shared__ __align__(16) T sX[Q * XT::LD], sY[Q * XT::LD];        // x and dy
    __shared__ __align__(16) T sB[Q * BT::LD], sC[Q * BT::LD];
    __shared__ __align__(16) T sM[NS * Q * MLD];                      // [term][j][i]
    __shared__ __align__(16) T sU[NS * SP * ULD];                     // [term][state][channel]
    __shared__ __align__(16) float sCum[Q], sDt[Q];
    __shared__ float sRow[NI][Q], sCol[NI][Q], sCd[4][Q], sE[4][Q], sDot[4], sDD[4];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane >> 4, l16 = lane & 15;
    const int slice = (int)(blockIdx.x % p.slices);
    const int64_t ng = blockIdx.x / p.slices;
    const int g = (int)(ng % p.G);
    const int64_t nc = ng / p.G, n = nc / p.K;
    const int c = (int)(nc - n * p.K), hpg = p.H / p.G;
    const int h_lo = slice * p.heads_per_slice, h_hi = min(hpg, h_lo + p.heads_per_slice);
    const int64_t len = seq_len(p.lengths, n, p.L), t0 = (int64_t)c * Q;
    const int rows = (int)max((int64_t)0, min((int64_t)Q, len - t0)), all_rows = (int)min((int64_t)Q, p.L - t0);
    const int64_t base = n * p.L + t0;
    const int64_t NK = (int64_t)p.N * p.K;

    f32x4 sc[TPW], ds[TPW], dB[NI][NTW], dC[NI][NTW];
    float cv[NI][NTW][4];
#pragma unroll
    for (int k = 0; k < TPW; ++k) sc[k] = ds[k] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int it = 0; it < NI; ++it)
#pragma unroll
        for (int k = 0; k < NTW; ++k) dB[it][k] = dC[it][k] = f32x4{0, 0, 0, 0};
    {
        BT bt, ct;
        bt.load((const T *)p.b + base * p.b_ld + (int64_t)g * p.S, p.b_ld, rows, p.S, p.vec);
        ct.load((const T *)p.c + base * p.c_ld + (int64_t)g * p.S, p.c_ld, rows, p.S, p.vec);
        bt.store(sB);
        ct.store(sC);
        for (int e = threadIdx.x; e < NS * Q * MLD; e += 256) sM[e] = (T)0.0f;
        for (int e = threadIdx.x; e < NI * Q; e += 256) sRow[0][e] = sCol[0][e] = 0.0f;
    }
    __syncthreads();
    // scores: rows i, column j in a lane
#pragma unroll
    for (int k = 0; k < TPW; ++k) {
        const int t = w + 4 * k;
        if (t < TRI) {
            int it, jt;
            tri_tile(t, it, jt);
#pragma unroll
            for (int ks = 0; ks < SP / 32; ++ks)
                sc[k] = mma(read_rows(sC, BT::LD, it * 16, ks * 32, lane), read_rows(sB, BT::LD, jt * 16, ks * 32, lane), sc[k]);
        }
    }
#pragma unroll
    for (int it = 0; it < NI; ++it)
#pragma unroll
        for (int k = 0; k < NTW; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                cv[it][k][r] = w + 4 * k < NT ? (float)sC[(it * 16 + q * 4 + r) * BT::LD + (w + 4 * k) * 16 + l16] : 0.0f;

    for (int hh = h_lo; hh < h_hi; ++hh) {
        const int h = g * hpg + hh;
        const float a = p.a[h], skip = p.d ? p.d[h] : 0.0f;
        float raw = 0.0f, dt = 0.0f, cum = 0.0f;
        float rs = 0.0f, cs = 0.0f, cd = 0.0f, ee = 0.0f, dot = 0.0f, dd = 0.0f;    // wave 0: per token, over the channel blocks
        if (w == 0) {
            if (lane < rows) raw = (float)((const T *)p.dt)[(base + lane) * p.dt_ld + h] + (p.dt_bias ? p.dt_bias[h] : 0.0f);
            chunk_decay(raw, lane < rows, a, p.softplus, lane, dt, cum);
        }
        for (int pb = 0; pb < p.NPB; ++pb) {
            const int pcols = min(kPB, p.P - pb * kPB);
            const int64_t xo = (int64_t)h * p.P + pb * kPB;
            XT xt, yt;
            xt.load((const T *)p.x + base * p.x_ld + xo, p.x_ld, rows, pcols, p.vec);
            yt.load((const T *)p.dy + base * p.dy_ld + xo, p.dy_ld, rows, pcols, p.vec);
            f32x4 h0[NTW][4], u[NTW][4];
            const int64_t bo = (((n * p.H + h) * p.NPB + pb) * p.K + c) * (SP * kPB);
            // behind the sequence x, dy and dt are zeros: any finite state will do
#pragma unroll
            for (int k = 0; k < NTW; ++k)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    h0[k][b] = u[k][b] = f32x4{0, 0, 0, 0};
                    if (w + 4 * k < NT && rows > 0) {
                        const int64_t o = bo + ((w + 4 * k) * 16 + l16) * kPB + b * 16 + q * 4;
                        h0[k][b] = *reinterpret_cast<const f32x4 *>(p.bound + o);
                        u[k][b] = *reinterpret_cast<const f32x4 *>(p.ubound + o);
                    }
                }
            float part = 0.0f;
#pragma unroll
            for (int k = 0; k < NTW; ++k)
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) part = fmaf(h0[k][b][r], u[k][b][r], part);
            part = wave_sum(part);
            __syncthreads();
            xt.store(sX);
            yt.store(sY);
            if (w == 0 && lane < Q) {
                sDt[lane] = dt;
                sCum[lane] = cum;
            }
            if (lane == 0) sDot[w] = part;
#pragma unroll
            for (int k = 0; k < NTW; ++k)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (w + 4 * k < NT)
                        write_split4<NS>(sU + ((w + 4 * k) * 16 + l16) * ULD + b * 16 + q * 4, SP * ULD, u[k][b]);
            __syncthreads();
            const float tot = sCum[Q - 1];
            // dP, M and dS, tile by tile; M goes to LDS transposed (rows j)
            float diag = 0.0f;
#pragma unroll
            for (int k = 0; k < TPW; ++k) {
                const int t = w + 4 * k;
                if (t < TRI) {
                    int it, jt;
                    tri_tile(t, it, jt);
                    f32x4 dp = {0, 0, 0, 0}, m, wr;
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
                        dp = mma(read_rows(sY, XT::LD, it * 16, ks * 32, lane), read_rows(sX, XT::LD, jt * 16, ks * 32, lane), dp);
                    const int i = it * 16 + q * 4, j = jt * 16 + l16;
                    const float cj = sCum[j], dj = sDt[j];
                    const f32x4 ci = *reinterpret_cast<const f32x4 *>(sCum + i);
                    float col = 0.0f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const bool in = i + r >= j;
                        const float dec = in ? exp2_fast(ci[r] - cj) : 0.0f;
                        if (i + r == j) diag += dp[r];
                        m[r] = in ? sc[k][r] * dec : 0.0f;
                        const float s = in ? dp[r] * dec * dj : 0.0f;
                        ds[k][r] += s;
                        wr[r] = s * sc[k][r];
                        col += wr[r];
                    }
                    write_split4<NS>(sM + j * MLD + i, Q * MLD, m);
                    col += __shfl_xor(col, 16);
                    col += __shfl_xor(col, 32);
                    if (q == 0) sCol[it][j] = col;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float s = row_sum(wr[r]);
                        if (l16 == 0) sRow[jt][i + r] = s;
                    }
                }
            }
            diag = wave_sum(diag);
            if (lane == 0) sDD[w] = diag;
            // dC and dB through the states at the borders
            float cdp[NI][4];
#pragma unroll
            for (int it = 0; it < NI; ++it)
#pragma unroll
                for (int r = 0; r < 4; ++r) cdp[it][r] = 0.0f;
#pragma unroll
            for (int k = 0; k < NTW; ++k) {
                if (w + 4 * k < NT) {
                    Split<T, NS> hs[2], us[2];
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = h0[k][2 * ks][e], v[4 + e] = h0[k][2 * ks + 1][e];
                        make_split(v, hs[ks]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = u[k][2 * ks][e], v[4 + e] = u[k][2 * ks + 1][e];
                        make_split(v, us[ks]);
                    }
#pragma unroll
                    for (int it = 0; it < NI; ++it) {
                        f32x4 ac = {0, 0, 0, 0}, ab = {0, 0, 0, 0};
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks) {
                            ac = mma_b(read_rows_stacked(sY, XT::LD, it * 16, ks * 32, lane), hs[ks], ac);
                            ab = mma_b(read_rows_stacked(sX, XT::LD, it * 16, ks * 32, lane), us[ks], ab);
                        }
                        const f32x4 ci = *reinterpret_cast<const f32x4 *>(sCum + it * 16 + q * 4);
                        const f32x4 di = *reinterpret_cast<const f32x4 *>(sDt + it * 16 + q * 4);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float v = ac[r] * exp2_fast(ci[r]);
                            dC[it][k][r] += v;
                            cdp[it][r] = fmaf(v, cv[it][k][r], cdp[it][r]);
                            dB[it][k][r] = fmaf(ab[r], exp2_fast(tot - ci[r]) * di[r], dB[it][k][r]);
                        }
                    }
                }
            }
#pragma unroll
            for (int it = 0; it < NI; ++it)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float s = row_sum(cdp[it][r]);
                    if (l16 == 0) sCd[w][it * 16 + q * 4 + r] = s;
                }
            __syncthreads();
            // dx, by channels
            {
                f32x4 dx[NI];
#pragma unroll
                for (int jt = 0; jt < NI; ++jt) dx[jt] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int ks = 0; ks < SP / 32; ++ks) {
                    frag uf[NS];
#pragma unroll
                    for (int m = 0; m < NS; ++m) uf[m] = read_cols(sU + m * SP * ULD, ULD, ks * 32, w * 16, lane);
#pragma unroll
                    for (int jt = 0; jt < NI; ++jt) {
                        const frag bf = read_rows(sB, BT::LD, jt * 16, ks * 32, lane);
#pragma unroll
                        for (int m = 0; m < NS; ++m) dx[jt] = mma(bf, uf[m], dx[jt]);
                    }
                }
#pragma unroll
                for (int jt = 0; jt < NI; ++jt) {
                    const f32x4 cj = *reinterpret_cast<const f32x4 *>(sCum + jt * 16 + q * 4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) dx[jt][r] *= exp2_fast(tot - cj[r]);
                }
#pragma unroll
                for (int ks = 0; ks < Q / 32; ++ks) {
                    const frag yf = read_cols(sY, XT::LD, ks * 32, w * 16, lane);
#pragma unroll
                    for (int jt = 0; jt < 2 * ks + 2; ++jt)
#pragma unroll
                        for (int m = 0; m < NS; ++m)
                            dx[jt] = mma(read_rows(sM + m * Q * MLD, MLD, jt * 16, ks * 32, lane), yf, dx[jt]);
                }
#pragma unroll
                for (int jt = 0; jt < NI; ++jt) {
                    const f32x4 dj = *reinterpret_cast<const f32x4 *>(sDt + jt * 16 + q * 4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int o = (jt * 16 + q * 4 + r) * XT::LD + w * 16 + l16;
                        const float s = row_sum((float)sX[o] * dx[jt][r]);
                        if (l16 == 0) sE[w][jt * 16 + q * 4 + r] = s;
                        sX[o] = (T)fmaf(skip, (float)sY[o], dj[r] * dx[jt][r]);     // this wave's own columns
                    }
                }
            }
            __syncthreads();
            XT::write(sX, (T *)p.dx + base * p.dx_ld + xo, p.dx_ld, all_rows, pcols, p.vec);
            if (w == 0) {
                if (lane < Q) {
#pragma unroll
                    for (int t = 0; t < NI; ++t) rs += sRow[t][lane], cs += sCol[t][lane];
#pragma unroll
                    for (int t = 0; t < 4; ++t) cd += sCd[t][lane], ee += sE[t][lane];
                }
                dot += (sDot[0] + sDot[1]) + (sDot[2] + sDot[3]);
                dd += (sDD[0] + sDD[1]) + (sDD[2] + sDD[3]);
            }
        }
        if (w == 0) {
            const float tot = wave_last(cum);
            const double before = (double)dt * ee - cs, behind = (double)rs - cs + cd;
            const double b1 = wave_prefix(before, lane), b2 = wave_prefix(behind, lane);
            const double all2 = __shfl(b2, 63);
            const float dl = (float)((b1 - before) + (all2 - b2 + behind) + (double)(exp2_fast(tot) * dot));
            float draw = fmaf(a, dl, ee);
            if (p.softplus) draw *= 1.0f / (1.0f + expf(-raw));
            if (lane >= rows) draw = 0.0f;
            if (lane < all_rows) ((T *)p.ddt)[(base + lane) * p.ddt_ld + h] = (T)draw;
            const float sa = wave_sum(dl * dt), sb = wave_sum(draw);
            if (lane == 0) {
                float *o = p.part_head + nc * p.H + h;
                o[0] = sa;
                o[NK * p.H] = sb;
                o[2 * NK * p.H] = dd;
            }
        }
    }
    // the parts of dB and dC inside the chunk, from the sum of dS over the heads
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TPW; ++k) {
        const int t = w + 4 * k;
        if (t < TRI) {
            int it, jt;
            tri_tile(t, it, jt);
            write_split4<NS>(sM + (jt * 16 + l16) * MLD + it * 16 + q * 4, Q * MLD, ds[k]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NTW; ++k) {
        const int nt = w + 4 * k;
        if (nt >= NT) continue;
#pragma unroll
        for (int ks = 0; ks < Q / 32; ++ks) {
            const frag bf = read_cols(sB, BT::LD, ks * 32, nt * 16, lane), cf = read_cols(sC, BT::LD, ks * 32, nt * 16, lane);
#pragma unroll
            for (int t = 0; t < NI; ++t)
#pragma unroll
                for (int m = 0; m < NS; ++m) {
                    const T *s = sM + m * Q * MLD;
                    if (t < 2 * ks + 2) dB[t][k] = mma(read_rows(s, MLD, t * 16, ks * 32, lane), cf, dB[t][k]);
                    if (t >= 2 * ks) dC[t][k] = mma(read_cols(s, MLD, ks * 32, t * 16, lane), bf, dC[t][k]);
                }
        }
        const int s = nt * 16 + l16;
        if (s >= p.S) continue;
#pragma unroll
        for (int t = 0; t < NI; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = t * 16 + q * 4 + r;
                if (row >= all_rows) continue;
                if (p.slices == 1) {
                    ((T *)p.db)[(base + row) * p.db_ld + g * p.S + s] = (T)dB[t][k][r];
                    ((T *)p.dc)[(base + row) * p.dc_ld + g * p.S + s] = (T)dC[t][k][r];
                } else {
                    const int64_t o = (((int64_t)slice * p.N * p.L + base + row) * p.G + g) * SP + s;
                    p.part_b[o] = dB[t][k][r];
                    p.part_c[o] = dC[t][k][r];
                }
            }
    }
}

// dB and dC from the head slices' parts, in their order
template <typename T, int SP> __global__ void __launch_bounds__(256) scan_reduce_bc_kernel(ScanParams p)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = (int64_t)p.N * p.L * p.G;
    if (id >= rows * SP) return;
    const int64_t rg = id / SP, row = rg / p.G;
    const int s = (int)(id - rg * SP), g = (int)(rg - row * p.G);
    if (s >= p.S) return;
    float b = 0.0f, c = 0.0f;
    for (int k = 0; k < p.slices; ++k) {
        b += p.part_b[k * rows * SP + id];
        c += p.part_c[k * rows * SP + id];
    }
    ((T *)p.db)[row * p.db_ld + g * p.S + s] = (T)b;
    ((T *)p.dc)[row * p.dc_ld + g * p.S + s] = (T)c;
}

// dA, ddt_bias and dD of a head: the chunks' parts in a fixed order
__global__ void __launch_bounds__(256) scan_reduce_heads_kernel(const float *part, float *da, float *dbias, float *dd,
                                                                int64_t NK, int H)
{
    __shared__ double red[256];
    const int which = blockIdx.x / H, h = blockIdx.x - which * H;
    float *out = which == 0 ? da : which == 1 ? dbias : dd;
    if (!out) return;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < NK; i += 256) s += part[(which * NK + i) * H + h];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) out[h] = (float)red[0];
}

// ---- one token -----------------------------------------------------------------
// The state is read and written once, 8 bytes for 5 flop: HBM bounds it, and at
// one sequence the launch does.  A wave takes kStepRows groups of channels; in a
// group 64 / LPR channels lie beside each other, LPR lanes with V neighbouring
// states each, so a wave's accesses are whole lines and y's sum is a few
// exchanges between lanes.
constexpr int kStepRows = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanParams p, int lpr, int blocks)
{
    constexpr int V = 4;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t nh = blockIdx.x / blocks, n = nh / p.H;
    const int blk = (int)(blockIdx.x - nh * blocks), h = (int)(nh - n * p.H), g = h / (p.H / p.G);
    const int per = 64 / lpr;                       // channels side by side in a wave
    const int s0 = (lane & (lpr - 1)) * V;
    const int ch0 = (blk * 4 + w) * kStepRows * per + lane / lpr;
    const T *bg = (const T *)p.b + n * p.b_ld + (int64_t)g * p.S, *cg = (const T *)p.c + n * p.c_ld + (int64_t)g * p.S;
    const T *xg = (const T *)p.x + n * p.x_ld + (int64_t)h * p.P;
    T *yg = (T *)p.y + n * p.y_ld + (int64_t)h * p.P;
    float st[kStepRows][V];
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) {
        const int ch = ch0 + k * per;
        const float *s = p.state + (nh * p.P + ch) * p.S + s0;
#pragma unroll
        for (int i = 0; i < V; ++i) st[k][i] = 0.0f;
        if (ch < p.P) {
            if (VEC) {
                if (s0 < p.S) load_f32<float, V>(s, st[k]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (s0 + i < p.S) st[k][i] = s[i];
            }
        }
    }
    float b[V], c[V], x[kStepRows];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        b[i] = s0 + i < p.S ? (float)bg[s0 + i] : 0.0f;
        c[i] = s0 + i < p.S ? (float)cg[s0 + i] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) x[k] = ch0 + k * per < p.P ? (float)xg[ch0 + k * per] : 0.0f;
    float dt = (float)((const T *)p.dt)[n * p.dt_ld + h] + (p.dt_bias ? p.dt_bias[h] : 0.0f);
    if (p.softplus) dt = softplus(dt);
    const float dec = exp2_fast(p.a[h] * dt * kLog2e), skip = p.d ? p.d[h] : 0.0f;
#pragma unroll
    for (int k = 0; k < kStepRows; ++k) {
        const int ch = ch0 + k * per;
        const float xd = x[k] * dt;
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            st[k][i] = fmaf(st[k][i], dec, xd * b[i]);
            y = fmaf(st[k][i], c[i], y);
        }
        for (int o = lpr >> 1; o > 0; o >>= 1) y += __shfl_xor(y, o);
        if (ch < p.P) {
            float *s = p.state_out + (nh * p.P + ch) * p.S + s0;
            if (VEC) {
                if (s0 < p.S) store_f32<float, V>(s, st[k]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (s0 + i < p.S) s[i] = st[k][i];
            }
            if (s0 == 0) yg[ch] = (T)fmaf(skip, x[k], y);
        }
    }
}

}  // namespace convfwd
