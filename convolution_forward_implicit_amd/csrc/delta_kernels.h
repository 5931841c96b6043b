// The gated delta rule, its gradient and its single-token step.
//
//   S' = e^{g_t} S,   y_t = v_t - S' k_t,   S = S' + beta_t y_t k_t^T,   o_t = scale S q_t
//
// per head, with a state S of P x S: a step replaces what the state holds under
// the key k_t by v_t, as far as the rate beta_t says.  Over a chunk of Q = 64
// tokens with c_i = sum_{j<=i} g_j and Gamma_ij = e^{c_i - c_j} (i >= j), every
// y depends on those before it by a triangular system, which is solved once
// for all channels (S_0 the state that the chunk starts from, i, j tokens):
//
//   T_ij = Gamma_ij k_i . k_j  (i > j)         N = (1 + T beta)^-1 T, strictly lower
//   Z = V - e^c K S_0^T                        Y = Z - N (beta Z),      U = beta Y
//   O = scale e^c Q S_0^T + M U                M_ij = scale Gamma_ij q_i . k_j  (i >= j)
//   S_Q = e^{c_Q} S_0 + sum_j e^{c_Q - c_j} U_j k_j^T
//
// (beta never divides, so it may be 0.)  With dO and the gradient R of S_Q:
//
//   dU = M^T dO + e^{c_Q - c} K R^T            E = dU - N^T (beta dU),  dV = beta E,  dbeta = E . Y
//   dS_0 = e^{c_Q} R + scale (e^c dO)^T Q - (e^c dV)^T K
//
// and the rest from S_0, R, Y and E of each chunk by itself (delta_grad_kernel).
// All exponents are differences of sums, at most 0 for g <= 0.  The sums are
// added in fp64, in powers of two; a g below -1e5 counts as that.  A difference is
// rounded to fp32 for its exponential, which is off by |c_i - c_j| 2^-24 of itself: 2^-20
// of a decay of e^-11, and less of the largest decay the further one has faded.  (fp32
// calls are 2.3e-7 off in 2-norm; plain fp32 operations with exponents in 64 bits 1.8e-7.)
//
// Numbers.  As in the scan, q, k and dO enter the bf16 matrix instructions as
// they are and what is computed on the way (states, Z, U, N, M) as the sum of three
// bf16 numbers: states come out with fp32's digits, and y with its own where its terms
// cancel.  (Two terms of what only y reads took 7% less of a prompt's time.)  fp32 calls
// run on the fp32 matrix instructions.
//
// delta_prepare_kernel does what a chunk can do without its state and leaves the
// operands of the matrix instructions in the workspace, each as the 64 lanes
// load it; the passes over the chunks follow in delta_chain.h.  The results of
// one product are the operand of the next as they stand: two results of 16 rows
// are an operand of a reduction over 32 (tokens 4q..4q+3 and 16+4q..16+4q+3 of
// lane group q), and the rows of K^T are taken in such an order that the states
// come out as 8 consecutive keys, which K's and Q's rows hold.
//
// Measured in bf16, heads of 128 channels and 128 keys, 4096 tokens: preparation 32 us
// (32 heads on 16 of keys; 95 MB, 3 TB/s, two workgroups a compute unit), y 119 us, 1.85
// us a chunk; gradient (16 heads) preparation 39, states 147, chunks 151 us (medians of a
// trace; the least 36, 139, 140).
#pragma once

#include "seq_frags.h"

namespace convfwd {

constexpr int kDQ = 64;         // tokens of a chunk
constexpr int kTri = 6;         // operands of a triangular 64 x 64 matrix: 16 rows x 32 columns each

struct DeltaParams {
    const void *q, *k, *v, *beta;
    const float *g, *state;
    const int32_t *lengths;
    void *y;
    float *state_out;
    int64_t q_ld, k_ld, v_ld, g_ld, beta_ld, y_ld;
    int64_t L;
    int N, H, P, G, S, K;       // K: chunks of a sequence
    int vec, slices, heads_per_slice, blocks;       // blocks: of 16 channels of a head
    float scale;
    char *keys, *heads;         // workspace: operands of a group's keys and of a head, by chunk
    // gradient
    const void *dy;
    const float *dstate_out;
    void *dq, *dk, *dv, *dbeta;
    float *dg, *dstate;
    int64_t dy_ld, dq_ld, dk_ld, dv_ld, dg_ld, dbeta_ld;
    int PP;                     // channels of a head in the workspace
    float *bound[2];            // [n, h][K][PP][SP]: the state in front of every chunk, the gradient of that behind it
    float *rows[2];             // [n, h][K * 64][PP]: Y and E
    float *part[2];             // [slice][N L][G][S]: dq and dk of a slice's heads
};

// ---- operands in the workspace -------------------------------------------------
template <typename T> constexpr int kFrag = 64 * 8 * (int)sizeof(T);
// K (4 x SP/32), Q (the same) and, for the gradient, K^T and Q^T (SP/16 x 2), k_i . k_j and q_i . k_j in fp32
template <typename T, int SP> constexpr int64_t frags_bytes(bool grad) { return (int64_t)(grad ? 4 : 2) * (SP / 8) * kFrag<T>; }
template <typename T, int SP> constexpr int64_t keys_bytes(bool grad)
{
    return frags_bytes<T, SP>(grad) + (grad ? 2 * kDQ * kDQ * 4 : 0);
}
// what a head adds, in terms: -N beta and M beta; gradient: -N beta, (-beta N)^T and M^T
template <typename T> constexpr int kN = 3;
template <> constexpr int kN<float> = 1;
struct ChunkScalars {
    float from_start[kDQ];      // e^{c_i}
    float beta[kDQ];
    float to_end[kDQ];          // e^{c_Q - c_i}
    float pad[kDQ];             // one load of 1 KB
    double cum[kDQ];            // c_i in powers of two; the gradient's
};
constexpr int kRows = 1024;     // bytes of ChunkScalars that the passes over the states read
// forward: ChunkScalars' first kilobyte, N, M; gradient: ChunkScalars, N, N^T, M^T
template <typename T> constexpr int64_t head_bytes(bool grad)
{
    return grad ? (int64_t)sizeof(ChunkScalars) + 3 * kN<T> * kTri * kFrag<T> : kRows + (int64_t)2 * kN<T> * kTri * kFrag<T>;
}

// The states of a chunk, and its rows, with 4 KB and 256 bytes between those of two
// chunks: workgroups that start together would all begin in the same memory channels
// (the gradient's chunks 140 -> 135 us).
constexpr int kApart = 1088;
constexpr int64_t states_floats(int PP, int SP) { return (int64_t)PP * SP + kApart; }
constexpr int64_t rows_floats(int PP) { return (int64_t)kDQ * PP + kApart; }

SEQ_DEV void put_frag(char *at, int lane, bf16x8 f) { reinterpret_cast<bf16x8 *>(at)[lane] = f; }
SEQ_DEV void put_frag(char *at, int lane, const Frag<float>::type &f)
{
    f32x4 *p = reinterpret_cast<f32x4 *>(at) + lane;
    p[0] = f32x4{f.v[0], f.v[1], f.v[2], f.v[3]};
    p[64] = f32x4{f.v[4], f.v[5], f.v[6], f.v[7]};
}
template <typename T> SEQ_DEV typename Frag<T>::type get_frag(const char *at, int lane)
{
    if constexpr (sizeof(T) == 2) {
        return reinterpret_cast<const bf16x8 *>(at)[lane];
    } else {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(at) + lane;
        const f32x4 a = p[0], b = p[64];
        Frag<float>::type f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f.v[e] = a[e], f.v[4 + e] = b[e];
        return f;
    }
}

// two results of 16 rows as an operand
template <typename T, int NS> SEQ_DEV void stack(f32x4 a, f32x4 b, Split<T, NS> &s)
{
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    make_split(v, s);
}

// a b of terms, up to those that the last term of the longer one is worth
template <typename T, int NA, int NB>
SEQ_DEV f32x4 mma_terms(const Split<T, NA> &a, const Split<T, NB> &b, f32x4 c)
{
    constexpr int most = NA > NB ? NA : NB;
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j < most) c = mma(a.f[i], b.f[j], c);
    return c;
}

// Operand (row tile i, columns 32 p ..) of a lower triangular matrix, and of an
// upper triangular one, among the six that are not all zeros.
SEQ_DEV constexpr int lower(int i, int p) { return i < 2 ? i : 2 * i - 2 + p; }
SEQ_DEV constexpr int upper(int i, int p) { return i < 2 ? 2 * i + p : 2 + i; }

// Columns k0 .. of 64 tokens as rows: tokens t0 + 4q .., t0 + 16 + 4q .. of key
// 32 s + 8 (r / 4) + 4 a + r % 4 for row r = lane % 16
SEQ_DEV bf16x8 read_keys(const bf16_t *t, int ld, int t0, int s, int a, int lane)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
    const bf16_t *p = t + (t0 + (lane >> 4) * 4 + ((lane & 15) >> 2)) * ld + 32 * s + 8 * (lane & 3) + 4 * a;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 16 * ld));
    return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
SEQ_DEV Frag<float>::type read_keys(const float *t, int ld, int t0, int s, int a, int lane)
{
    const int r = lane & 15;
    const float *p = t + (t0 + (lane >> 4) * 4) * ld + 32 * s + 8 * (r >> 2) + 4 * a + (r & 3);
    Frag<float>::type f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = p[e * ld], f.v[4 + e] = p[(16 + e) * ld];
    return f;
}

// ---- what a chunk can do without its state ---------------------------------------
template <typename T, int SP, bool GRAD> struct PrepareShared {
    static constexpr int LD = Tile<T, kDQ, SP>::LD;
    static constexpr int TL = kDQ + 4;
    struct Rows {
        T k[kDQ * LD], q[kDQ * LD];
    };
    struct Solve {              // when the rows have been read
        float t[GRAD ? 2 : 1][kDQ * TL];        // [j][i]: T transposed; gradient: then N and M, transposed
        float inv[4][16][20];   // [block][j][m]: the inverse of a block of 1 + beta T on the diagonal, transposed
    };
    static constexpr int BYTES = sizeof(Rows) > sizeof(Solve) ? sizeof(Rows) : sizeof(Solve);
    __align__(16) char at[BYTES];
    double cum[4][kDQ];         // every wave's own
    float beta[4][kDQ];
};

// One chunk of one group: 4 waves, wave I owns the rows 16 I .. of T, N and M.
// Everything is formed transposed (result rows j, columns i), so that the rows
// of the operands come out as they are stored.  The inverse is that of forward
// substitution by blocks of 16 (stable also where keys repeat): row blocks of N
// do not depend on each other, N_IJ = (T_IJ - sum_{J<M<=I} N_IM beta T_MJ) (1 +
// beta T_JJ)^-1, on the fp32 matrix instructions.
template <typename T, int SP, bool GRAD>
__global__ void __launch_bounds__(256, SP <= 128 ? 2 : 1) delta_prepare_kernel(DeltaParams p)
{
    typedef PrepareShared<T, SP, GRAD> Shared;
    constexpr int LD = Shared::LD, TL = Shared::TL, KS = SP / 32;
    __shared__ Shared sh;
    typename Shared::Rows &in = *reinterpret_cast<typename Shared::Rows *>(sh.at);
    typename Shared::Solve &so = *reinterpret_cast<typename Shared::Solve *>(sh.at);
    const int lane = threadIdx.x & 63, w = wave_id(), l16 = lane & 15, q4 = (lane >> 4) * 4;
    const int64_t chunk = blockIdx.x / ((int64_t)p.G * p.slices);        // n K + c
    const int gs = (int)(blockIdx.x - chunk * p.G * p.slices), grp = gs / p.slices, slice = gs - grp * p.slices;
    const int64_t n = chunk / p.K, t0 = (chunk - n * p.K) * kDQ, len = seq_len(p.lengths, n, p.L);
    if (t0 >= len) return;
    const int live = (int)(len - t0 < kDQ ? len - t0 : kDQ);
    const int per = p.H / p.G, h0 = grp * per + slice * p.heads_per_slice;
    const int h1 = min(h0 + p.heads_per_slice, (grp + 1) * per);
    const int64_t row = n * p.L + t0 + (lane < live ? lane : 0);
    float g = p.g[row * p.g_ld + h0], rate = (float)((const T *)p.beta)[row * p.beta_ld + h0];
    {
        Tile<T, kDQ, SP> a, b;
        a.load((const T *)p.k + (n * p.L + t0) * p.k_ld + (int64_t)grp * p.S, p.k_ld, live, p.S, p.vec);
        b.load((const T *)p.q + (n * p.L + t0) * p.q_ld + (int64_t)grp * p.S, p.q_ld, live, p.S, p.vec);
        a.store(in.k);
        b.store(in.q);
    }
    __syncthreads();
    // k_j . k_i and k_j . q_i: rows j of tile J, columns i of tile w
    f32x4 kk[4], kq[4];
#pragma unroll
    for (int J = 0; J < 4; ++J) kk[J] = kq[J] = f32x4{0, 0, 0, 0};
    char *out = p.keys + (chunk * p.G + grp) * keys_bytes<T, SP>(GRAD);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const typename Frag<T>::type bk = read_rows(in.k, LD, 16 * w, 32 * s, lane), bq = read_rows(in.q, LD, 16 * w, 32 * s, lane);
        if (slice == 0) {
            put_frag(out + (w * KS + s) * kFrag<T>, lane, bk);
            put_frag(out + (4 * KS + w * KS + s) * kFrag<T>, lane, bq);
        }
#pragma unroll
        for (int J = 0; J < 4; ++J) {
            if (J > w) continue;
            const typename Frag<T>::type a = read_rows(in.k, LD, 16 * J, 32 * s, lane);
            kk[J] = mma(a, bk, kk[J]);
            kq[J] = mma(a, bq, kq[J]);
        }
    }
    if (GRAD && slice == 0)
        for (int f = w; f < 4 * KS; f += 4) {       // (s, a, pair of token tiles)
            put_frag(out + (8 * KS + f) * kFrag<T>, lane, read_keys(in.k, LD, 32 * (f & 1), f >> 2, f >> 1 & 1, lane));
            put_frag(out + (12 * KS + f) * kFrag<T>, lane, read_keys(in.q, LD, 32 * (f & 1), f >> 2, f >> 1 & 1, lane));
        }
    const int i = 16 * w + l16;
    if (GRAD && slice == 0) {
        f32x4 *dots = reinterpret_cast<f32x4 *>(out + frags_bytes<T, SP>(true)) + i * (kDQ / 4) + (lane >> 4);
#pragma unroll
        for (int J = 0; J < 4; ++J)
            if (J <= w) dots[4 * J] = kk[J], dots[kDQ * kDQ / 4 + 4 * J] = kq[J];
    }
    for (int h = h0; h < h1; ++h) {
        char *at = p.heads + (chunk * p.H + h) * head_bytes<T>(GRAD);
        {
            const bool on = lane < live;
            const double step = (double)(g < -1e5f ? -1e5f : g) * 1.4426950408889634074;
            const float beta = on ? rate : 0.0f;
            const double cum = wave_prefix(on ? step : 0.0), end = wave_last(cum);
            if (h + 1 < h1) {       // the next head's
                g = p.g[row * p.g_ld + h + 1];
                rate = (float)((const T *)p.beta)[row * p.beta_ld + h + 1];
            }
            sh.cum[w][lane] = cum;
            sh.beta[w][lane] = beta;
            if (w == 0) {
                ChunkScalars *cs = reinterpret_cast<ChunkScalars *>(at);
                cs->from_start[lane] = exp2_fast((float)cum);
                cs->to_end[lane] = exp2_fast((float)(end - cum));
                cs->beta[lane] = beta;
                if (GRAD) cs->cum[lane] = cum;
            }
        }
        at += GRAD ? (int64_t)sizeof(ChunkScalars) : kRows;
        __syncthreads();        // the rows, or the last head's T, have been read
        f32x4 tt[4], mm[4];
        {
            const double ci = sh.cum[w][i];
#pragma unroll
            for (int J = 0; J < 4; ++J) {
                tt[J] = mm[J] = f32x4{0, 0, 0, 0};
                if (J > w) continue;
                const f32x4 beta = *reinterpret_cast<const f32x4 *>(&sh.beta[w][16 * J + q4]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 16 * J + q4 + r;
                    const float decay = j <= i ? exp2_fast((float)(ci - sh.cum[w][j])) : 0.0f;
                    tt[J][r] = j < i ? kk[J][r] * decay : 0.0f;
                    mm[J][r] = j <= i ? kq[J][r] * decay * p.scale * (GRAD ? 1.0f : beta[r]) : 0.0f;
                    so.t[0][j * TL + i] = tt[J][r];
                }
            }
        }
        if constexpr (!GRAD) {
#pragma unroll
            for (int P = 0; P < 2; ++P) {
                if (2 * P > w) continue;
                Split<T, kN<T>> s;
                stack(mm[2 * P], mm[2 * P + 1], s);
#pragma unroll
                for (int e = 0; e < kN<T>; ++e) put_frag(at + (kTri * kN<T> + lower(w, P) * kN<T> + e) * kFrag<T>, lane, s.f[e]);
            }
        }
        // column l16 of (1 + beta T_ww)^-1, by forward substitution in this wave's own block
        {
            float x[16];
#pragma unroll
            for (int m = 0; m < 16; ++m) x[m] = m == l16 ? 1.0f : 0.0f;
#pragma unroll
            for (int l = 0; l < 15; ++l) {
#pragma unroll
                for (int m4 = (l + 1) / 4 * 4; m4 < 16; m4 += 4) {
                    const f32x4 col = *reinterpret_cast<const f32x4 *>(&so.t[0][(16 * w + l) * TL + 16 * w + m4]) *
                                      *reinterpret_cast<const f32x4 *>(&sh.beta[w][16 * w + m4]);
#pragma unroll
                    for (int m = m4; m < m4 + 4; ++m)
                        if (m > l) x[m] = fmaf(-col[m - m4], x[l], x[m]);
                }
            }
            if (lane < 16) {
#pragma unroll
                for (int m = 0; m < 16; m += 4)
                    *reinterpret_cast<f32x4 *>(&so.inv[w][l16][m]) = f32x4{x[m], x[m + 1], x[m + 2], x[m + 3]};
            }
        }
        __syncthreads();
        f32x4 nn[4], nb[4];     // N, and -beta N, transposed
#pragma unroll
        for (int J = 3; J >= 0; --J) {
            nn[J] = nb[J] = f32x4{0, 0, 0, 0};
            if (J > w) continue;
            f32x4 rhs = tt[J];
#pragma unroll
            for (int M = 3; M > J; --M) {
                if (M > w) continue;
                const f32x4 a = *reinterpret_cast<const f32x4 *>(&so.t[0][(16 * J + l16) * TL + 16 * M + q4]);
#pragma unroll
                for (int r = 0; r < 4; ++r) rhs = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], nb[M][r], rhs, 0, 0, 0);
            }
            const f32x4 a = *reinterpret_cast<const f32x4 *>(&so.inv[J][l16][q4]);
#pragma unroll
            for (int r = 0; r < 4; ++r) nn[J] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], rhs[r], nn[J], 0, 0, 0);
            nb[J] = nn[J] * *reinterpret_cast<const f32x4 *>(&sh.beta[w][16 * J + q4]) * -1.0f;
        }
#pragma unroll
        for (int P = 0; P < 2; ++P) {
            if (2 * P > w) continue;
            Split<T, kN<T>> s;
            stack(nb[2 * P], nb[2 * P + 1], s);
#pragma unroll
            for (int e = 0; e < kN<T>; ++e) put_frag(at + (lower(w, P) * kN<T> + e) * kFrag<T>, lane, s.f[e]);
        }
        if constexpr (GRAD) {
            at += kTri * kN<T> * kFrag<T>;
            __syncthreads();
#pragma unroll
            for (int J = 0; J < 4; ++J)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    so.t[0][(16 * J + q4 + r) * TL + i] = nn[J][r];
                    so.t[1][(16 * J + q4 + r) * TL + i] = mm[J][r];
                }
            __syncthreads();
#pragma unroll
            for (int which = 0; which < 2; ++which) {
#pragma unroll
                for (int P = 0; P < 2; ++P) {
                    if (2 * P + 1 < w) continue;
                    f32x4 v[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        v[e] = *reinterpret_cast<const f32x4 *>(&so.t[which][i * TL + 32 * P + 16 * e + q4]);
                        if (!which) v[e] = v[e] * *reinterpret_cast<const f32x4 *>(&sh.beta[w][32 * P + 16 * e + q4]) * -1.0f;
                    }
                    Split<T, kN<T>> s;
                    stack(v[0], v[1], s);
#pragma unroll
                    for (int e = 0; e < kN<T>; ++e) put_frag(at + (upper(w, P) * kN<T> + e) * kFrag<T>, lane, s.f[e]);
                }
                at += kTri * kN<T> * kFrag<T>;
            }
        }
    }
}

// ---- the state, chunk by chunk -----------------------------------------------------
// Workgroups in XCD order: neighbours share operands, and so an L2.
SEQ_DEV int64_t unit_of(int64_t block, int64_t units)
{
    const int64_t per = (units + 7) / 8;
    return (block & 7) * per + (block >> 3);
}

// ---- the gradient of a chunk ---------------------------------------------------------
// From the state S in front of the chunk, the gradient R of that behind it, Y and E
// (U = beta Y, dV = beta E; D and W lower triangular, W strictly):
//
//   D = dO U^T,  W = dV U^T,   pair_ij = D_ij M_ij - W_ij T_ij
//   dq = scale (e^c dO S + (D o Gamma) K)
//   dk = scale (D o Gamma)^T Q - e^c dV S + e^{c_Q - c} U R - (W o Gamma + its transpose) K
//   dg_t = sum_{i>=t} (scale e^c dO S . q - e^c dV S . k)_i + sum_{j<t} (e^{c_Q - c} U R . k)_j
//        + sum_{j<t<=i} pair_ij + e^{c_Q} <S, R>
//
// (every path of dg_t crosses the decay of token t; a pair counts as its row less
// its column, the same number in fp64 twice, so that what cancels leaves nothing).
// One workgroup takes one chunk of a slice of a group's heads; a wave owns CT
// blocks of 16 keys, in the order of K^T's operands, and reads S and R itself, a step
// ahead: no other wave needs them.  dO, dV and U go through LDS, split into their terms
// once, their rows fetched a block of channels ahead.
//
// 1024 chunks of 128 channels and keys in bf16 take 140 us and more: 290 KB a chunk, 2.1 TB/s.  One
// workgroup of eight waves fits a compute unit (256 registers a thread, 147 KB of LDS).
// A workgroup that went from chunk to chunk and loaded the next one's first rows beside
// the last phases of this one took 147 us, its registers spilled; the products of keys
// and queries, taken here once a chunk instead of from the preparation, 150 (against 139 in turn).
// 128 keys put 12 bytes a lane in scratch memory (fp32 76); with 256 the sums of three products
// leave too few registers and it is some 650.
template <typename T, int SP> struct GradShape {
    static constexpr int NW = SP <= 64 ? 4 : 8;                      // waves
    static constexpr int CT = SP / 16 < NW ? 1 : SP / 16 / NW;
    static constexpr int PB = 64;                                    // channels at a time
    static constexpr int TT = (10 + NW - 1) / NW;                    // triangular tiles of a wave
    static constexpr int LD = PB + Frag<T>::PAD, ML = kDQ + Frag<T>::PAD;
    static constexpr int NL = kN<T>;                                 // terms of D o Gamma and W o Gamma
};
template <typename T, int SP> struct GradShared {
    typedef GradShape<T, SP> G;
    T dy[kDQ * G::LD], dv[kN<T>][kDQ * G::LD], u[kN<T>][kDQ * G::LD];
    T low[G::NL][kDQ * G::ML], sym[G::NL][kDQ * G::ML];
    float from_start[kDQ], to_end[kDQ], beta[kDQ];
    double cum[kDQ];
    double row[4][kDQ], col[4][kDQ], front[G::NW][kDQ], behind[G::NW][kDQ], across[G::NW];
};

// tile t of the ten on and below the diagonal of 4 x 4
SEQ_DEV void triangle(int t, int &i, int &j)
{
    i = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
    j = t - i * (i + 1) / 2;
}

// Column col0 + lane % 16 of 64 rows, rows k0 + 4q .. and k0 + 16 + 4q ..
SEQ_DEV bf16x8 read_cols_stacked(const bf16_t *t, int ld, int k0, int col0, int lane)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
    const bf16_t *p = t + (k0 + (lane >> 4) * 4 + ((lane & 15) >> 2)) * ld + col0 + (lane & 3) * 4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 16 * ld));
    return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
SEQ_DEV Frag<float>::type read_cols_stacked(const float *t, int ld, int k0, int col0, int lane)
{
    const float *p = t + (k0 + (lane >> 4) * 4) * ld + col0 + (lane & 15);
    Frag<float>::type f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = p[e * ld], f.v[4 + e] = p[(16 + e) * ld];
    return f;
}

// an element a lane's number of bytes from an address that all lanes share: no
// register pairs for addresses
template <typename X> SEQ_DEV X *lane_at(X *base, uint32_t bytes)
{
    return reinterpret_cast<X *>(reinterpret_cast<uintptr_t>(base) + bytes);
}

// element (row, col) of a matrix held as terms
template <typename T, int NS, int ALL> SEQ_DEV void put_terms(T (&m)[NS][ALL], int at, float v)
{
#pragma unroll
    for (int e = 0; e < NS; ++e) {
        const T t = (T)v;
        m[e][at] = t;
        v -= (float)t;
    }
}

template <typename T, int SP> __global__ void __launch_bounds__(SP <= 64 ? 256 : 512) delta_grad_kernel(DeltaParams p)
{
    typedef GradShape<T, SP> G;
    constexpr int NW = G::NW, CT = G::CT, PB = G::PB, TT = G::TT, LD = G::LD, ML = G::ML, NL = G::NL, KS = SP / 32;
    constexpr int kRowsAtOnce = NW * 4, RI = kDQ / kRowsAtOnce;     // 16 threads take a row of PB channels
    __shared__ __align__(16) GradShared<T, SP> sh;
    const int lane0 = threadIdx.x & 63, w = wave_id();
    const int lane = lane0, l16 = lane & 15, q = lane >> 4;
    // a phase takes its lane anew, so that its LDS addresses (beyond an instruction's offset) are not all computed
    // before the loop over the heads and held
#define NEW_LANE const int lane = fresh_vector(lane0), l16 = lane & 15, q = lane >> 4, q4 = q * 4; (void)lane, (void)l16, (void)q, (void)q4
    const bool cols = w * CT < SP / 16;                                  // a wave that has keys
    const int tri = NW - 1 - w;                                          // the others first
    const int64_t chunk = blockIdx.x / ((int64_t)p.G * p.slices);        // n K + c
    const int gs = (int)(blockIdx.x - chunk * p.G * p.slices), grp = gs / p.slices, slice = gs - grp * p.slices;
    const int64_t n = chunk / p.K, c = chunk - n * p.K, t0 = c * kDQ, len = seq_len(p.lengths, n, p.L);
    const int live = (int)(len - t0 < 0 ? 0 : len - t0 < kDQ ? len - t0 : kDQ);
    const int all = (int)(p.L - t0 < kDQ ? p.L - t0 : kDQ);              // rows of the outputs
    const int per = p.H / p.G, h0 = grp * per + slice * p.heads_per_slice;
    const int h1 = min(h0 + p.heads_per_slice, (grp + 1) * per);
    const int64_t row0 = n * p.L + t0;
    const int key0 = 8 * (l16 >> 2) + (l16 & 3);       // key of this lane's column in block (s, a): 32 s + 4 a + key0
    if (live < all) {           // rows behind the sequence; where none is in front there is nothing else
        for (int e = threadIdx.x; e < (all - live) * (h1 - h0); e += NW * 64) {
            const int64_t row = row0 + live + e / (h1 - h0);
            const int h = h0 + e % (h1 - h0);
            p.dg[row * p.dg_ld + h] = 0.0f;
            ((T *)p.dbeta)[row * p.dbeta_ld + h] = (T)0.0f;
        }
        const int64_t wide = (int64_t)(h1 - h0) * p.P;
        for (int64_t e = threadIdx.x; e < (all - live) * wide; e += NW * 64)
            ((T *)p.dv)[(row0 + live + e / wide) * p.dv_ld + (int64_t)h0 * p.P + e % wide] = (T)0.0f;
        for (int e = threadIdx.x; e < (all - live) * p.S; e += NW * 64) {
            const int64_t row = row0 + live + e / p.S;
            const int key = e % p.S;
            if (p.slices == 1) {
                ((T *)p.dq)[row * p.dq_ld + (int64_t)grp * p.S + key] = (T)0.0f;
                ((T *)p.dk)[row * p.dk_ld + (int64_t)grp * p.S + key] = (T)0.0f;
            } else {
                const int64_t at = (((int64_t)slice * p.N * p.L + row) * p.G + grp) * p.S + key;
                p.part[0][at] = p.part[1][at] = 0.0f;
            }
        }
    }
    const int64_t part = (((int64_t)slice * p.N * p.L + row0) * p.G + grp) * p.S;
    const uint32_t part_step = (uint32_t)(p.G * p.S) * 4;
    const char *keys = p.keys + (chunk * p.G + grp) * keys_bytes<T, SP>(true);
    const char *kt = keys + 8 * KS * kFrag<T>, *qt = kt + 4 * KS * kFrag<T>;
    // the upper triangles stay zero
    for (int e = threadIdx.x; e < kDQ * ML; e += NW * 64)
#pragma unroll
        for (int x = 0; x < NL; ++x) sh.low[x][e] = (T)0.0f;
    const int my_row = threadIdx.x >> 4;
    const uint32_t dy_step = (uint32_t)p.dy_ld * (uint32_t)sizeof(T), dv_step = (uint32_t)p.dv_ld * (uint32_t)sizeof(T);
    // The next block of channels: Y, E and dO's bits.  Rows and channels that there are none of lie behind the buffers'
    // ends and come as zeros: a load under a branch would be waited for in it.
    constexpr uint32_t NOWHERE = 0x80000000u;
    f32x4 ry[RI], re[RI];
    uint32_t rd[RI][4];
    auto rows_of = [&](const void *t, int64_t ld, int h) {
        return __builtin_amdgcn_make_buffer_rsrc((T *)const_cast<void *>(t) + row0 * ld + (int64_t)h * p.P, 0,
                                                 (int)(((live - 1) * ld + p.P) * (int64_t)sizeof(T)), 0x00020000);
    };
    auto load_rows = [&](int h, int p0) {
        const int pc = p0 + 4 * l16;
        const int64_t at = ((n * p.H + h) * p.K + c) * rows_floats(p.PP);
        const __amdgpu_buffer_rsrc_t gy = __builtin_amdgcn_make_buffer_rsrc(p.rows[0] + at, 0, live * p.PP * 4, 0x00020000);
        const __amdgpu_buffer_rsrc_t ge = __builtin_amdgcn_make_buffer_rsrc(p.rows[1] + at, 0, live * p.PP * 4, 0x00020000);
        const __amdgpu_buffer_rsrc_t gd = rows_of(p.dy, p.dy_ld, h);
#pragma unroll
        for (int e = 0; e < RI; ++e) {
            const int row = my_row + e * kRowsAtOnce;
            const uint32_t o = pc < p.PP ? (uint32_t)(row * p.PP + pc) * 4 : NOWHERE;
            ry[e] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(gy, o, 0, 0));
            re[e] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ge, o, 0, 0));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t d = pc + i < p.P ? (uint32_t)row * dy_step + (uint32_t)(pc + i) * (uint32_t)sizeof(T) : NOWHERE;
                if constexpr (sizeof(T) == 4) rd[e][i] = __builtin_amdgcn_raw_buffer_load_b32(gd, d, 0, 0);
                else rd[e][i] = __builtin_amdgcn_raw_buffer_load_b16(gd, d, 0, 0);
            }
        }
    };
    // a head's factors of token `lane`; the first wave gives them to the others
    float grow_of, fade_of, beta_of;
    double cum_of;
    auto load_scalars = [&](int h) {
        const ChunkScalars *cs = reinterpret_cast<const ChunkScalars *>(p.heads + (chunk * p.H + h) * head_bytes<T>(true));
        grow_of = cs->from_start[lane];
        fade_of = cs->to_end[lane];
        beta_of = cs->beta[lane];
        cum_of = cs->cum[lane];
    };
    float sv[CT][8], rv[CT][8];         // the next 32 channels of S and R
    auto load_states = [&](int h, int p0) {
        if (!cols) return;
        const int64_t at = ((n * p.H + h) * p.K + c) * states_floats(p.PP, SP) + (int64_t)p0 * SP;
#pragma unroll
        for (int x = 0; x < CT; ++x) {
            const int b = w * CT + x;
            const uint32_t o = (uint32_t)(8 * q * SP + 32 * (b >> 1) + 4 * (b & 1) + key0) * 4;
            const float *gs = lane_at(p.bound[0] + at, o), *gr = lane_at(p.bound[1] + at, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) sv[x][i] = gs[i * SP], rv[x][i] = gr[i * SP];
        }
    };
    if (live > 0) {
        load_scalars(h0);
        load_rows(h0, 0);
        load_states(h0, 0);
    }
    for (int h = h0; h < (live > 0 ? h1 : h0); ++h) {
        __syncthreads();
        if (w == 0) {
            sh.from_start[lane] = grow_of;
            sh.to_end[lane] = fade_of;
            sh.beta[lane] = beta_of;
            sh.cum[lane] = cum_of;
        }
        if (h + 1 < h1) load_scalars(h + 1);
        const __amdgpu_buffer_rsrc_t gv = rows_of(p.dv, p.dv_ld, h);
        f32x4 by[CT][4], old[CT][4], nw[CT][4], dm[TT], wm[TT];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int x = 0; x < CT; ++x) by[x][t] = old[x][t] = nw[x][t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < TT; ++t) dm[t] = wm[t] = f32x4{0, 0, 0, 0};
        float db[RI];
#pragma unroll
        for (int e = 0; e < RI; ++e) db[e] = 0.0f;
        double across = 0.0;
        for (int p0 = 0; p0 < p.PP; p0 += PB) {
            NEW_LANE;
            const int my_row = 4 * w + q;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < RI; ++e) {
                const int row = my_row + e * kRowsAtOnce, pc = p0 + 4 * l16;
                const float beta = sh.beta[row];
#pragma unroll
                for (int i = 0; i < 4; ++i) db[e] = fmaf(re[e][i], ry[e][i], db[e]);
                const f32x4 dv = re[e] * beta;
                f32x4 dy;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t to = pc + i < p.P ? (uint32_t)row * dv_step + (uint32_t)(pc + i) * (uint32_t)sizeof(T) : NOWHERE;
                    const uint32_t bits = sizeof(T) == 4 ? rd[e][i] : rd[e][i] << 16;
                    dy[i] = __builtin_bit_cast(float, bits);
                    if constexpr (sizeof(T) == 4)
                        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (float)dv[i]), gv, to, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)dv[i]), gv, to, 0, 0);
                }
                const int at = row * LD + 4 * l16;
                write_split4<1>(sh.dy + at, 0, dy);
                write_split4<kN<T>>(sh.dv[0] + at, kDQ * LD, dv);
                write_split4<kN<T>>(sh.u[0] + at, kDQ * LD, ry[e] * beta);
            }
            if (p0 + PB < p.PP) load_rows(h, p0 + PB);
            else if (h + 1 < h1) load_rows(h + 1, 0);
            __syncthreads();
            // one step after the other, and one row tile: all of their reads at once leave no registers
#pragma unroll 1
            for (int s = 0; s < PB / 32; ++s) {
                if (p0 + 32 * s >= p.PP) break;
                NEW_LANE;
                if (cols) {
                    Split<T, kN<T>> ss[CT], rs[CT];
#pragma unroll
                    for (int x = 0; x < CT; ++x) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) across = fma((double)sv[x][i], (double)rv[x][i], across);
                        make_split(sv[x], ss[x]);
                        make_split(rv[x], rs[x]);
                    }
                    if (p0 + 32 * (s + 1) < p.PP) load_states(h, p0 + 32 * (s + 1));
                    else if (h + 1 < h1) load_states(h + 1, 0);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        Split<T, 1> a;
                        Split<T, kN<T>> d, u;
                        a.f[0] = read_rows(sh.dy, LD, 16 * t, 32 * s, lane);
#pragma unroll
                        for (int e = 0; e < kN<T>; ++e) {
                            d.f[e] = read_rows(sh.dv[e], LD, 16 * t, 32 * s, lane);
                            u.f[e] = read_rows(sh.u[e], LD, 16 * t, 32 * s, lane);
                        }
#pragma unroll
                        for (int x = 0; x < CT; ++x) {
                            by[x][t] = mma_terms(a, ss[x], by[x][t]);
                            old[x][t] = mma_terms(d, ss[x], old[x][t]);
                            nw[x][t] = mma_terms(u, rs[x], nw[x][t]);
                        }
                        in_order();
                    }
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (tri + t * NW >= 10) continue;
                    int it, jt;
                    triangle(tri + t * NW, it, jt);
                    Split<T, 1> a;
                    Split<T, kN<T>> d, u;
                    a.f[0] = read_rows(sh.dy, LD, 16 * it, 32 * s, lane);
#pragma unroll
                    for (int e = 0; e < kN<T>; ++e) {
                        d.f[e] = read_rows(sh.dv[e], LD, 16 * it, 32 * s, lane);
                        u.f[e] = read_rows(sh.u[e], LD, 16 * jt, 32 * s, lane);
                    }
                    dm[t] = mma_terms(a, u, dm[t]);
                    wm[t] = mma_terms(d, u, wm[t]);
                    in_order();
                }
            }
        }
        // K^T and Q^T, under way while the pairs are summed
        typename Frag<T>::type kf[CT][2], qf[CT][2];
        if (cols) {
            NEW_LANE;
#pragma unroll
            for (int x = 0; x < CT; ++x)
#pragma unroll
                for (int P = 0; P < 2; ++P) {
                    kf[x][P] = get_frag<T>(kt + ((w * CT + x) * 2 + P) * kFrag<T>, lane);
                    qf[x][P] = get_frag<T>(qt + ((w * CT + x) * 2 + P) * kFrag<T>, lane);
                }
        }
        // and k_i . k_j, q_i . k_j
        f32x4 kk[TT], qk[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (tri + t * NW >= 10) continue;
            NEW_LANE;
            int it, jt;
            triangle(tri + t * NW, it, jt);
            const float *dots = lane_at(reinterpret_cast<const float *>(keys + frags_bytes<T, SP>(true)),
                                        (uint32_t)((16 * it + q4) * kDQ + 16 * jt + l16) * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) kk[t][r] = dots[r * kDQ], qk[t][r] = dots[kDQ * kDQ + r * kDQ];
        }
        in_order();
        // dbeta: the 16 threads of a row
#pragma unroll
        for (int e = 0; e < RI; ++e) {
            NEW_LANE;
            const int my_row = 4 * w + q;
            float v = db[e];
            for (int o = 8; o > 0; o >>= 1) v += __shfl_xor(v, o);
            const int row = my_row + e * kRowsAtOnce;
            if (l16 == 0 && row < live)
                *lane_at((T *)p.dbeta + row0 * p.dbeta_ld + h, (uint32_t)row * (uint32_t)p.dbeta_ld * (uint32_t)sizeof(T)) = (T)v;
        }
        // pairs of tokens
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (tri + t * NW >= 10) continue;
            NEW_LANE;
            int it, jt;
            triangle(tri + t * NW, it, jt);
            f32x4 pair;
            const int j = 16 * jt + l16;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * it + q4 + r;
                const float decay = i >= j ? exp2_fast((float)(sh.cum[i] - sh.cum[j])) : 0.0f;
                const float lo = i >= j ? dm[t][r] * (decay * p.scale) : 0.0f, be = i > j ? wm[t][r] * decay : 0.0f;
                pair[r] = i > j ? lo * qk[t][r] - be * kk[t][r] : 0.0f;      // a token's pair with itself crosses no decay
                put_terms(sh.low, i * ML + j, lo);
                if (i >= j) {
                    put_terms(sh.sym, i * ML + j, -be);
                    put_terms(sh.sym, j * ML + i, -be);
                }
            }
            const double sum = row_sum4<double>(pair, lane);
            if ((l16 & 3) == 0) sh.row[jt][16 * it + q4 + (l16 >> 2)] = sum;
            double down = ((double)pair[0] + (double)pair[1]) + ((double)pair[2] + (double)pair[3]);
            down += __shfl_xor(down, 16);
            down += __shfl_xor(down, 32);
            if (q == 0) sh.col[it][j] = down;
            in_order();
        }
        // what the states in front and behind give (dq and dk stand where by and old did), and its part in dg
        auto &dq = by, &dk = old;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (!cols) break;
            NEW_LANE;
            double front = 0.0, behind = 0.0;
            const f32x4 grow = *reinterpret_cast<const f32x4 *>(sh.from_start + 16 * t + q4);
            const f32x4 fade = *reinterpret_cast<const f32x4 *>(sh.to_end + 16 * t + q4);
#pragma unroll
            for (int x = 0; x < CT; ++x) {
                by[x][t] = by[x][t] * (grow * p.scale);
                old[x][t] = old[x][t] * grow;
                nw[x][t] = nw[x][t] * fade;
                f32x4 a, b;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float kv = frag_get(kf[x][t >> 1], 4 * (t & 1) + r), qv = frag_get(qf[x][t >> 1], 4 * (t & 1) + r);
                    a[r] = by[x][t][r] * qv - old[x][t][r] * kv;
                    b[r] = nw[x][t][r] * kv;
                }
                front += row_sum4<double>(a, lane);
                behind += row_sum4<double>(b, lane);
                dk[x][t] = nw[x][t] - old[x][t];
                in_order();
            }
            if ((l16 & 3) == 0) {
                sh.front[w][16 * t + q4 + (l16 >> 2)] = front;
                sh.behind[w][16 * t + q4 + (l16 >> 2)] = behind;
            }
        }
        for (int o = 32; o > 0; o >>= 1) across += __shfl_xor(across, o);
        if (lane == 0) sh.across[w] = across;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < CT; ++x)
#pragma unroll
            for (int P = 0; P < 2; ++P) {
                if (!cols) continue;
                NEW_LANE;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
#pragma unroll
                    for (int e = 0; e < NL; ++e) {
                        if (P <= t / 2) dq[x][t] = mma(read_rows_stacked(sh.low[e], ML, 16 * t, 32 * P, lane), kf[x][P], dq[x][t]);
                        dk[x][t] = mma(read_rows_stacked(sh.sym[e], ML, 16 * t, 32 * P, lane), kf[x][P], dk[x][t]);
                        if (P >= t / 2) dk[x][t] = mma(read_cols_stacked(sh.low[e], ML, 32 * P, 16 * t, lane), qf[x][P], dk[x][t]);
                    }
                    in_order();
                }
            }
        if (w == 0) {
            NEW_LANE;
            double d = 0.0, b = 0.0, whole = 0.0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e <= lane >> 4) d += sh.row[e][lane];
                if (e >= lane >> 4) d -= sh.col[e][lane];
            }
#pragma unroll
            for (int e = 0; e < NW; ++e)
                if (e * CT < SP / 16) d += sh.front[e][lane], b += sh.behind[e][lane], whole += sh.across[e];
            if (lane >= live) d = b = 0.0;
            const double upto = wave_prefix(d), sum = wave_last(upto), before = wave_prefix(b) - b;
            const double dg = (sum - upto + d) + before + (double)sh.from_start[kDQ - 1] * whole;
            const double step = lane > 0 ? sh.cum[lane] - sh.cum[lane - 1] : sh.cum[0];
            // no gradient by a decay that is zero
            if (lane < live) p.dg[(row0 + lane) * p.dg_ld + h] = exp2_fast((float)step) == 0.0f ? 0.0f : (float)dg;
        }
        // dq and dk: the sums over the slice's heads wait in the workspace, where a lane finds its own again (held in
        // registers they would leave the products above too few), and behind the last head go to the outputs, or stay
        // for the sum over the slices
        const bool out = h + 1 == h1 && p.slices == 1;
#pragma unroll
        for (int x = 0; x < CT; ++x) {
            NEW_LANE;
            const int b = w * CT + x, key = 32 * (b >> 1) + 4 * (b & 1) + 8 * (l16 >> 2) + (l16 & 3);
            if (!cols || key >= p.S) continue;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * t + q4 + r;
                    if (row >= live) continue;
                    float *sq = lane_at(p.part[0] + part, (uint32_t)row * part_step + (uint32_t)key * 4);
                    float *sk = lane_at(p.part[1] + part, (uint32_t)row * part_step + (uint32_t)key * 4);
                    const float vq = dq[x][t][r] + (h > h0 ? *sq : 0.0f), vk = dk[x][t][r] + (h > h0 ? *sk : 0.0f);
                    if (out) {
                        const uint32_t k = (uint32_t)key * (uint32_t)sizeof(T);
                        *lane_at((T *)p.dq + row0 * p.dq_ld + (int64_t)grp * p.S, (uint32_t)row * (uint32_t)p.dq_ld * (uint32_t)sizeof(T) + k) = (T)vq;
                        *lane_at((T *)p.dk + row0 * p.dk_ld + (int64_t)grp * p.S, (uint32_t)row * (uint32_t)p.dk_ld * (uint32_t)sizeof(T) + k) = (T)vk;
                    } else {
                        *sq = vq;
                        *sk = vk;
                    }
                }
        }
    }
}
#undef NEW_LANE

// dq and dk from the slices' sums, always in the same order
template <typename T> __global__ void __launch_bounds__(256) delta_reduce_kernel(DeltaParams p)
{
    const int64_t rows = (int64_t)p.N * p.L, width = (int64_t)p.G * p.S, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= rows * width) return;
    const int64_t row = e / width, col = e - row * width;
    float q = 0.0f, k = 0.0f;
    for (int s = 0; s < p.slices; ++s) {
        q += p.part[0][s * rows * width + e];
        k += p.part[1][s * rows * width + e];
    }
    ((T *)p.dq)[row * p.dq_ld + col] = (T)q;
    ((T *)p.dk)[row * p.dk_ld + col] = (T)k;
}

// ---- one token -----------------------------------------------------------------------
// With s = S k, o = S q of the old state and d = k . q, all in one pass over it:
// y = v - e^g s, the output scale (e^g o + beta d y), the new state e^g S + beta y k^T.
// A lane holds four keys of kDeltaRows channels; `lpr` lanes share a channel.  64 sequences
// of 32 heads, 128 x 128: 56 us, 4.8 TB/s of states read and written.
constexpr int kDeltaRows = 4;

template <typename T, bool VEC> __global__ void __launch_bounds__(256) delta_step_kernel(DeltaParams p, int lpr, int blocks)
{
    constexpr int V = 4, R = kDeltaRows;
    const int lane = threadIdx.x & 63, w = wave_id();
    const int64_t nh = blockIdx.x / blocks, n = nh / p.H;
    const int blk = (int)(blockIdx.x - nh * blocks), h = (int)(nh - n * p.H), grp = h / (p.H / p.G);
    const int per = 64 / lpr;                       // channels side by side in a wave
    const int s0 = (lane & (lpr - 1)) * V;
    const int ch0 = (blk * 4 + w) * R * per + lane / lpr;
    const T *kg = (const T *)p.k + n * p.k_ld + (int64_t)grp * p.S, *qg = (const T *)p.q + n * p.q_ld + (int64_t)grp * p.S;
    const T *vg = (const T *)p.v + n * p.v_ld + (int64_t)h * p.P;
    T *yg = (T *)p.y + n * p.y_ld + (int64_t)h * p.P;
    float st[R][V], k[V], q[V], v[R];
#pragma unroll
    for (int e = 0; e < R; ++e) {
        const int ch = ch0 + e * per;
        const float *s = p.state + (nh * p.P + ch) * p.S + s0;
#pragma unroll
        for (int i = 0; i < V; ++i) st[e][i] = 0.0f;
        if (ch < p.P) {
            if (VEC) {
                if (s0 < p.S) load_f32<float, V>(s, st[e]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (s0 + i < p.S) st[e][i] = s[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        k[i] = s0 + i < p.S ? (float)kg[s0 + i] : 0.0f;
        q[i] = s0 + i < p.S ? (float)qg[s0 + i] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < R; ++e) v[e] = ch0 + e * per < p.P ? (float)vg[ch0 + e * per] : 0.0f;
    const float fade = expf(p.g[n * p.g_ld + h]), beta = (float)((const T *)p.beta)[n * p.beta_ld + h];
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) d = fmaf(k[i], q[i], d);
    for (int o = lpr >> 1; o > 0; o >>= 1) d += __shfl_xor(d, o);
#pragma unroll
    for (int e = 0; e < R; ++e) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) a = fmaf(st[e][i], k[i], a), b = fmaf(st[e][i], q[i], b);
        for (int o = lpr >> 1; o > 0; o >>= 1) a += __shfl_xor(a, o), b += __shfl_xor(b, o);
        const int ch = ch0 + e * per;
        const float u = beta * fmaf(-fade, a, v[e]);
#pragma unroll
        for (int i = 0; i < V; ++i) st[e][i] = fmaf(st[e][i], fade, u * k[i]);
        if (ch < p.P) {
            float *s = p.state_out + (nh * p.P + ch) * p.S + s0;
            if (VEC) {
                if (s0 < p.S) stream_f32<float, V>(s, st[e]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (s0 + i < p.S) s[i] = st[e][i];
            }
            if (s0 == 0) yg[ch] = (T)(p.scale * fmaf(fade, b, u * d));
        }
    }
}

}  // namespace convfwd
