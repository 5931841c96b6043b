// The gated delta rule over a prompt, on pairs of fp16 numbers.
//
// Numbers.  A matrix operand is the sum of fp16 numbers: q and k of bf16 tensors
// are one each (8 bits of 11), what is computed on the way and fp32 tensors two,
// the rounding and the rounding of what it left, 2^-24 of the value together.
// fp16 has few exponents, so each column of an operand's reduction (a channel of a
// state, of Z, of U; a token's key; all of N and of M) is scaled by a power of two
// that brings its largest element to 2^14..2^15; what is 2^-29 of that counts as
// zero.  Products are added in fp32 and scaled back.  Three bf16 terms hold as many
// digits without a scale, but take 3 products for 2 and 6 for 3 (two computed
// operands) and 11 vector instructions for a pair of values where these take 6.  y of
// bf16 tensors takes one fp16 term of the state, of M and of Y, 2^-12 of the value
// where y's own rounding is 2^-8.
#pragma once

#include "delta_kernels.h"
#include "igemm_dma.h"

namespace convfwd {

typedef _Float16 f16_t;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <int N> struct Terms {
    f16x8 f[N];
};
SEQ_DEV f32x4 mma(f16x8 a, f16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
template <int NA, int NB> SEQ_DEV f32x4 mma(const Terms<NA> &a, const Terms<NB> &b, f32x4 c)
{
    constexpr int most = NA > NB ? NA : NB;
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j < most) c = mma(a.f[i], b.f[j], c);
    return c;
}

// A power of two that brings the largest of some values, given by its bits without the
// sign, to 2^14..2^15, and its inverse; an infinity or a NaN stays one.
struct Scale {
    float f, inv;
};
SEQ_DEV Scale scale_of(uint32_t bits)
{
    const uint32_t e = bits >> 23, c = e < 15 ? 15 : e > 254 ? 254 : e;
    return {__builtin_bit_cast(float, (268 - c) << 23), __builtin_bit_cast(float, (c - 14) << 23)};
}
SEQ_DEV uint32_t max_bits(uint32_t a, uint32_t b) { return a > b ? a : b; }
SEQ_DEV uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
// the largest of a result's channel in registers ..
template <int N> SEQ_DEV uint32_t largest(const f32x4 (&v)[N])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(v[i][r]));
    return abs_bits(m);
}
// .. and of the four groups of lanes that share it
SEQ_DEV uint32_t channel_max(uint32_t m)
{
    const auto a = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    const uint32_t b = max_bits(a[0], a[1]);
    const auto c = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    return max_bits(c[0], c[1]);
}

template <int N> SEQ_DEV void split(const float (&v)[8], float f, Terms<N> &t)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const f16x2 hi = __builtin_convertvector((f32x2{v[e] * f, v[e + 1] * f}), f16x2);
        t.f[0][e] = hi[0], t.f[0][e + 1] = hi[1];
        if constexpr (N > 1) {
            const f32x2 left = {fmaf(v[e], f, -(float)hi[0]), fmaf(v[e + 1], f, -(float)hi[1])};
            const f16x2 lo = __builtin_convertvector(left, f16x2);
            t.f[1][e] = lo[0], t.f[1][e + 1] = lo[1];
        }
    }
}
// two results of 16 rows as an operand
template <int N> SEQ_DEV void stack(f32x4 a, f32x4 b, float f, Terms<N> &t)
{
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    split(v, f, t);
}

// ---- the workspace -----------------------------------------------------------------
// Operands of 16 rows x 32 columns: 1 KB, lane l's 16 bytes at 16 l.
constexpr int kOp = 1024;
template <typename T> constexpr int kIn = sizeof(T) == 2 ? 1 : 2;      // terms of q, k; of what y of that type takes

// K and Q of a group's chunk: [term][row tile][32 keys]
template <typename T, int SP> constexpr int kKeysBytes = kIn<T> * (SP / 8) * kOp;
// what multiplies the rows of a chunk, scales of its keys among it (ek, eq: the exponents of row i)
struct ChunkRows {
    float gk[kDQ];              // e^{c_i} 2^ek             of K S in Z
    float uk[kDQ];              // beta_i e^{c_Q - c_i} 2^ek     of Y in the state
    float gq[kDQ];              // scale e^{c_i} 2^eq       of Q S in y
    float mq[kDQ];              // 2^eq 2^em                of M Y in y
    float sn, total;            // 2^en, e^{c_Q}
    float pad[254];
};
static_assert(sizeof(ChunkRows) == 2 * kOp, "whole loads");
// a head's chunk: -N beta of two terms, ChunkRows, M beta
constexpr int kHeadRows = kTri * 2 * kOp, kHeadM = kHeadRows + (int)sizeof(ChunkRows);
template <typename T> constexpr int kHeadBytes = kHeadM + kTri * kIn<T> * kOp;

// Rows 16 t .. of a matrix of SP columns in operands, this lane's 16 bytes
SEQ_DEV f16x8 get_op(const char *at, int lane) { return reinterpret_cast<const f16x8 *>(at)[lane]; }
template <int N> SEQ_DEV void get_terms(const char *at, int apart, int lane, Terms<N> &t)
{
#pragma unroll
    for (int e = 0; e < N; ++e) t.f[e] = get_op(at + e * apart, lane);
}
// The transpose of the operands at `at` (tokens 32 P .. of [row tile][KS], in LDS): keys
// 32 s + 8 (r / 4) + 4 a + r % 4 in row r, tokens 32 P + 4q .. and 32 P + 16 + 4q ..
template <int KS> SEQ_DEV f16x8 get_transposed(const char *at, int P, int s, int a, int lane)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
    const int i = lane & 15;
    const char *p = at + (2 * P * KS + s) * kOp + ((i & 3) * 16 + (lane >> 4) * 4 + (i >> 2)) * 16 + 8 * a;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + KS * kOp));
    return __builtin_bit_cast(f16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ---- what a chunk can do without its state -------------------------------------------
template <typename T, int SP> struct PairsShared {
    static constexpr int TL = kDQ + 4;
    char k[kKeysBytes<T, SP>], q[kKeysBytes<T, SP>];
    float ek[kDQ], eq[kDQ];     // 2^ek, 2^eq of the rows
    float t[kDQ * TL];          // [j][i]: T transposed
    float inv[4][16][20];       // [block][j][m]: the inverse of a block of 1 + beta T on the diagonal, transposed
    float beta[kDQ];
    uint32_t most[2][4];        // of N and of M, by wave
    double cum[kDQ];
};

// a tile's rows, scaled and split, as operands in LDS; the rows' scales
template <typename T, int SP> SEQ_DEV void put_keys(const Tile<T, kDQ, SP> &tile, char *out, float *scales)
{
    typedef Tile<T, kDQ, SP> Rows;
    constexpr int VE = Rows::VE, CV = Rows::CV;
#pragma unroll
    for (int e = 0; e < Rows::NV; ++e) {
        const int row = (int)threadIdx.x / CV + e * Rows::kStep, col = Rows::column();
        float v[VE];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const uint32_t word = tile.v[e][sizeof(T) == 4 ? i : i / 2];
            v[i] = __builtin_bit_cast(float, sizeof(T) == 4 ? word : i & 1 ? word & 0xffff0000u : word << 16);
            m = max_bits(m, abs_bits(v[i]));
        }
        for (int o = CV / 2; o > 0; o >>= 1) m = max_bits(m, (uint32_t)__shfl_xor((int)m, o));
        const Scale s = scale_of(m);
        if (!Rows::mine()) continue;
        if (col == 0) scales[row] = s.inv;
        // 8 columns are a lane's 16 bytes
        char *at = out + (row / 16 * (SP / 32) + col / 32) * kOp + (col % 32 / 8 * 16 + row % 16) * 16 + col % 8 * 2;
        typedef _Float16 f16v __attribute__((ext_vector_type(VE)));
        f16v hi, lo;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            hi[i] = (f16_t)(v[i] * s.f);
            lo[i] = (f16_t)fmaf(v[i], s.f, -(float)hi[i]);
        }
        *reinterpret_cast<f16v *>(at) = hi;
        if constexpr (kIn<T> > 1) *reinterpret_cast<f16v *>(at + SP / 8 * kOp) = lo;
    }
}

// delta_prepare_kernel's work on pairs
template <typename T, int SP> __global__ void __launch_bounds__(256) delta_chunks_kernel(DeltaParams p)
{
    typedef PairsShared<T, SP> Shared;
    constexpr int TL = Shared::TL, KS = SP / 32, NI = kIn<T>, KEYS = kKeysBytes<T, SP>;
    __shared__ __align__(16) Shared sh;
    const int lane = threadIdx.x & 63, w = wave_id(), l16 = lane & 15, q4 = (lane >> 4) * 4;
    const int64_t chunk = blockIdx.x / ((int64_t)p.G * p.slices);        // n K + c
    const int gs = (int)(blockIdx.x - chunk * p.G * p.slices), grp = gs / p.slices, slice = gs - grp * p.slices;
    const int64_t n = chunk / p.K, t0 = (chunk - n * p.K) * kDQ, len = seq_len(p.lengths, n, p.L);
    if (t0 >= len) return;
    const int live = (int)(len - t0 < kDQ ? len - t0 : kDQ);
    {
        Tile<T, kDQ, SP> a, b;
        a.load((const T *)p.k + (n * p.L + t0) * p.k_ld + (int64_t)grp * p.S, p.k_ld, live, p.S, p.vec);
        b.load((const T *)p.q + (n * p.L + t0) * p.q_ld + (int64_t)grp * p.S, p.q_ld, live, p.S, p.vec);
        put_keys(a, sh.k, sh.ek);
        put_keys(b, sh.q, sh.eq);
    }
    __syncthreads();
    if (slice == 0) {
        char *at = p.keys + (chunk * p.G + grp) * 2 * KEYS;
        for (int o = threadIdx.x * 16; o < KEYS; o += 256 * 16) {
            *reinterpret_cast<f32x4 *>(at + o) = *reinterpret_cast<const f32x4 *>(sh.k + o);
            *reinterpret_cast<f32x4 *>(at + KEYS + o) = *reinterpret_cast<const f32x4 *>(sh.q + o);
        }
    }
    // k_j . k_i and k_j . q_i / 2^eq: rows j of tile J, columns i of tile w
    const int i = 16 * w + l16;
    f32x4 kk[4], kq[4];
    {
        Terms<NI> bk[KS], bq[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            get_terms(sh.k + (w * KS + s) * kOp, 4 * KS * kOp, lane, bk[s]);
            get_terms(sh.q + (w * KS + s) * kOp, 4 * KS * kOp, lane, bq[s]);
        }
        const float eki = sh.ek[i];
#pragma unroll
        for (int J = 0; J < 4; ++J) {
            kk[J] = kq[J] = f32x4{0, 0, 0, 0};
            if (J > w) continue;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                Terms<NI> a;
                get_terms(sh.k + (J * KS + s) * kOp, 4 * KS * kOp, lane, a);
                kk[J] = mma(a, bk[s], kk[J]);
                kq[J] = mma(a, bq[s], kq[J]);
            }
            const f32x4 ekj = *reinterpret_cast<const f32x4 *>(sh.ek + 16 * J + q4);
            kk[J] = kk[J] * (ekj * eki);
            kq[J] = kq[J] * ekj;
        }
    }
    const int per = p.H / p.G, h0 = grp * per + slice * p.heads_per_slice;
    const int h1 = min(h0 + p.heads_per_slice, (grp + 1) * per);
    for (int h = h0; h < h1; ++h) {
        char *at = p.heads + (chunk * p.H + h) * kHeadBytes<T>;
        ChunkRows *rows = reinterpret_cast<ChunkRows *>(at + kHeadRows);
        // every wave has the sums itself; wave 0 leaves them for all
        float beta;
        double cum, end;
        {
            const int64_t row = n * p.L + t0 + lane;
            const float g = lane < live ? p.g[row * p.g_ld + h] : 0.0f;
            beta = lane < live ? (float)((const T *)p.beta)[row * p.beta_ld + h] : 0.0f;
            cum = wave_prefix((double)(g < -1e5f ? -1e5f : g));
            end = wave_last(cum);
            if (w == 0) {
                sh.cum[lane] = cum;
                sh.beta[lane] = beta;
            }
        }
        __syncthreads();
        f32x4 tt[4], mm[4], bj[4];
        const double ci = sh.cum[i];
#pragma unroll
        for (int J = 0; J < 4; ++J) {
            bj[J] = *reinterpret_cast<const f32x4 *>(sh.beta + 16 * J + q4);
            tt[J] = mm[J] = f32x4{0, 0, 0, 0};
            if (J > w) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = 16 * J + q4 + r;
                const float decay = j <= i ? expf((float)(ci - sh.cum[j])) : 0.0f;
                tt[J][r] = j < i ? kk[J][r] * decay : 0.0f;
                mm[J][r] = j <= i ? kq[J][r] * decay * p.scale * bj[J][r] : 0.0f;
                sh.t[j * TL + i] = tt[J][r];
            }
        }
        // column l16 of (1 + beta T_ww)^-1, by forward substitution on this wave's own block
        {
            float x[16];
#pragma unroll
            for (int m = 0; m < 16; ++m) x[m] = m == l16 ? 1.0f : 0.0f;
            const f32x4 bw[4] = {*reinterpret_cast<const f32x4 *>(sh.beta + 16 * w), *reinterpret_cast<const f32x4 *>(sh.beta + 16 * w + 4),
                                 *reinterpret_cast<const f32x4 *>(sh.beta + 16 * w + 8), *reinterpret_cast<const f32x4 *>(sh.beta + 16 * w + 12)};
#pragma unroll
            for (int l = 0; l < 15; ++l) {
                f32x4 col[4];
#pragma unroll
                for (int m = (l + 1) / 4; m < 4; ++m)
                    col[m] = *reinterpret_cast<const f32x4 *>(sh.t + (16 * w + l) * TL + 16 * w + 4 * m) * bw[m];
#pragma unroll
                for (int m = l + 1; m < 16; ++m) x[m] = fmaf(-col[m / 4][m % 4], x[l], x[m]);
            }
            if (lane < 16) {
#pragma unroll
                for (int m = 0; m < 16; m += 4)
                    *reinterpret_cast<f32x4 *>(&sh.inv[w][l16][m]) = f32x4{x[m], x[m + 1], x[m + 2], x[m + 3]};
            }
        }
        __syncthreads();
        f32x4 nb[4];            // -beta N, transposed
#pragma unroll
        for (int J = 3; J >= 0; --J) {
            nb[J] = f32x4{0, 0, 0, 0};
            if (J > w) continue;
            f32x4 rhs = tt[J], nn = {0, 0, 0, 0};
#pragma unroll
            for (int M = 3; M > J; --M) {
                if (M > w) continue;
                const f32x4 a = *reinterpret_cast<const f32x4 *>(sh.t + (16 * J + l16) * TL + 16 * M + q4);
#pragma unroll
                for (int r = 0; r < 4; ++r) rhs = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], nb[M][r], rhs, 0, 0, 0);
            }
            const f32x4 a = *reinterpret_cast<const f32x4 *>(&sh.inv[J][l16][q4]);
#pragma unroll
            for (int r = 0; r < 4; ++r) nn = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], rhs[r], nn, 0, 0, 0);
            nb[J] = nn * bj[J] * -1.0f;
        }
        // one scale for all of N, one for all of M
        uint32_t most_n = largest(nb), most_m = largest(mm);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            most_n = max_bits(most_n, (uint32_t)__shfl_xor((int)most_n, o));
            most_m = max_bits(most_m, (uint32_t)__shfl_xor((int)most_m, o));
        }
        if (lane == 0) sh.most[0][w] = most_n, sh.most[1][w] = most_m;
        __syncthreads();
        const Scale sn = scale_of(max_bits(max_bits(sh.most[0][0], sh.most[0][1]), max_bits(sh.most[0][2], sh.most[0][3])));
        const Scale sm = scale_of(max_bits(max_bits(sh.most[1][0], sh.most[1][1]), max_bits(sh.most[1][2], sh.most[1][3])));
#pragma unroll
        for (int P = 0; P < 2; ++P) {
            if (2 * P > w) continue;
            Terms<2> a;
            Terms<NI> b;
            stack(nb[2 * P], nb[2 * P + 1], sn.f, a);
            stack(mm[2 * P], mm[2 * P + 1], sm.f, b);
#pragma unroll
            for (int e = 0; e < 2; ++e) reinterpret_cast<f16x8 *>(at + (e * kTri + lower(w, P)) * kOp)[lane] = a.f[e];
#pragma unroll
            for (int e = 0; e < NI; ++e) reinterpret_cast<f16x8 *>(at + kHeadM + (e * kTri + lower(w, P)) * kOp)[lane] = b.f[e];
        }
        if (w == 0) {
            const float grow = expf((float)cum), ek = sh.ek[lane], eq = sh.eq[lane];
            rows->gk[lane] = grow * ek;
            rows->uk[lane] = beta * expf((float)(end - cum)) * ek;
            rows->gq[lane] = p.scale * grow * eq;
            rows->mq[lane] = eq * sm.inv;
            if (lane == 63) rows->sn = sn.inv, rows->total = grow;
        }
        __syncthreads();        // cum, beta and t are the next head's
    }
}

// ---- the state, chunk by chunk ---------------------------------------------------------
// A workgroup takes NS x 16 channels of a head.  Of its 2 NS waves the first NS hold
// a state of 16 channels and all keys each, and take it from chunk to chunk; nothing
// of a chunk leaves their registers but what y needs: the state's terms and Y go
// through LDS to the other NS waves, which compute the y of a chunk while the next is
// under way, and bring the operands that the state waves share (K and N) into LDS a
// chunk ahead.  Q and M have one reader each and go to its registers.  One barrier a
// chunk.
template <typename T, int SP, int NS> struct StateShared {
    static constexpr int NI = kIn<T>, KS = SP / 32;
    static constexpr int KN = kKeysBytes<T, SP> + kHeadM;
    static constexpr int NB = 2 * KN + 2 * NS * (NI * KS * kOp + 4 * kOp + 64) <= 160 * 1024 ? 2 : 1;   // chunks of operands
    struct Exchange {
        char s[NI * KS * kOp];          // the state's terms, as it enters the chunk
        f32x4 y[4][64];
        float inv[16];                  // the scales of the state's channels
    };
    __align__(16) char kn[NB][KN];
    Exchange x[2][NS];
};

// KB kilobytes of memory to LDS, by NS waves.  The loads are written out: the compiler,
// which cannot see what they write, would wait for them before any read of LDS.
template <int KB, int NS> SEQ_DEV void fetch(const char *from, char *to, int wave, int lane)
{
    const i32x4_t buf = uniform_rsrc(buffer_rsrc(from, KB * kOp));
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)to);
#pragma unroll
    for (int e = 0; e < KB; e += NS) {
        const uint32_t b = (uint32_t)(e + wave) * kOp;
        uint32_t saved;
        if (KB % NS == 0 || e + wave < KB)
            asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
                         : "=&s"(saved) : "s"(at + b), "v"(lane * 16), "s"(buf), "s"(b) : "memory");
    }
}
// The 16 rows that a lane of a result holds (16 t + 4q + r of column `ch`) of 64 rows of
// a tensor, from row `first`: rows at `rows` and behind, and columns that are not `mine`,
// come as zeros and are not written.
template <typename T> struct LaneRows {
    __amdgpu_buffer_rsrc_t buf;
    uint32_t at, step;
    SEQ_DEV LaneRows(const void *g, int64_t ld, int64_t first, int rows, int P, int ch, int lane)
    {
        const int64_t bytes = rows > 0 ? ((rows - 1) * ld + P) * (int64_t)sizeof(T) : 0;
        buf = __builtin_amdgcn_make_buffer_rsrc((T *)const_cast<void *>(g) + first * ld, 0, (int)bytes, 0x00020000);
        step = (uint32_t)ld * (uint32_t)sizeof(T);
        at = ch < P ? (uint32_t)((lane >> 4) * 4) * step + (uint32_t)ch * (uint32_t)sizeof(T) : 0x80000000u;
    }
    SEQ_DEV uint32_t offset(int e) const { return at + (uint32_t)(16 * (e / 4) + e % 4) * step; }
    SEQ_DEV uint32_t bits(int e) const      // of an element, as a float's
    {
        if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b32(buf, offset(e), 0, 0);
        else return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(buf, offset(e), 0, 0) << 16;
    }
    SEQ_DEV void put(int e, float v) const
    {
        if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), buf, offset(e), 0, kStream);
        else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)v), buf, offset(e), 0, kStream);
    }
};
// The workgroup's waves meet; LDS writes are done, loads may be under way.
SEQ_DEV void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <typename T, int SP, int NS> __global__ void __launch_bounds__(128 * NS) delta_state_kernel(DeltaParams p)
{
    typedef StateShared<T, SP, NS> Shared;
    constexpr int NI = kIn<T>, KS = SP / 32, KEYS = kKeysBytes<T, SP>, NB = Shared::NB;
    __shared__ Shared sh;
    const int blocks = (p.blocks + NS - 1) / NS;
    const int64_t units = (int64_t)p.N * p.H * blocks, unit = unit_of(blockIdx.x, units);
    if (unit >= units) return;
    const int lane = threadIdx.x & 63, w = wave_id(), l16 = lane & 15, q4 = (lane >> 4) * 4;
    const int64_t nh = unit / blocks, n = nh / p.H;
    const int h = (int)(nh - n * p.H), grp = h / (p.H / p.G), s_wave = w < NS ? w : w - NS;
    const int ch = ((int)(unit - nh * blocks) * NS + s_wave) * 16 + l16;
    const bool mine = ch < p.P;
    const int chc = mine ? ch : 0;              // a channel that is there
    const int64_t len = seq_len(p.lengths, n, p.L);
    const int live = (int)((len + kDQ - 1) / kDQ);
    const char *keys = p.keys + (n * p.K * p.G + grp) * 2 * KEYS, *heads = p.heads + (n * p.K * p.H + h) * kHeadBytes<T>;
    const int64_t keys_step = (int64_t)p.G * 2 * KEYS, head_step = (int64_t)p.H * kHeadBytes<T>;
    auto fetch_chunk = [&](int c) {
        fetch<KEYS / kOp, NS>(keys + c * keys_step, sh.kn[c % NB], s_wave, lane);
        fetch<kHeadM / kOp, NS>(heads + c * head_step, sh.kn[c % NB] + KEYS, s_wave, lane);
    };
    if (w < NS) {
        f32x4 st[SP / 16];
        load_state<SP>(p.state + (nh * p.P + chc) * p.S, p.state && mine, p.S, lane, st);
        uint32_t v[16];                         // the next chunk's
        auto load_v = [&](int c) {
            const int64_t t0 = (int64_t)c * kDQ;
            const LaneRows<T> rows((const T *)p.v + (int64_t)h * p.P, p.v_ld, n * p.L + t0, (int)(len - t0 < kDQ ? len - t0 : kDQ), p.P,
                                   ch, lane);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = rows.bits(e);
        };
        if (live > 0) load_v(0);
        meet();
        for (int c = 0; c <= live; ++c) {
            if (NB == 1) meet();       // the operands of this chunk are there
            if (c < live) {
                const char *kn = sh.kn[c % NB], *nn = kn + KEYS;
                const ChunkRows *rows = reinterpret_cast<const ChunkRows *>(nn + kHeadRows);
                typename Shared::Exchange &x = sh.x[c & 1][w];
                f32x4 acc[4], z[4], gk[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) acc[t] = f32x4{0, 0, 0, 0}, gk[t] = *reinterpret_cast<const f32x4 *>(rows->gk + 16 * t + q4);
                Terms<NI> ks[2][4];             // K's operands of a step ahead
#pragma unroll
                for (int t = 0; t < 4; ++t) get_terms(kn + t * KS * kOp, 4 * KS * kOp, lane, ks[0][t]);
                const Scale ss = scale_of(channel_max(largest(st)));
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    Terms<2> sp;
                    stack(st[2 * s], st[2 * s + 1], ss.f, sp);
#pragma unroll
                    for (int e = 0; e < NI; ++e) reinterpret_cast<f16x8 *>(x.s + (e * KS + s) * kOp)[lane] = sp.f[e];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        if (s + 1 < KS) get_terms(kn + (t * KS + s + 1) * kOp, 4 * KS * kOp, lane, ks[(s + 1) & 1][t]);
                        acc[t] = mma(ks[s & 1][t], sp, acc[t]);
                    }
                }
                if (lane < 16) x.inv[lane] = ss.inv;
                Terms<2> ns[kTri];
#pragma unroll
                for (int f = 0; f < kTri; ++f) get_terms(nn + f * kOp, kTri * kOp, lane, ns[f]);
                f32x4 uk[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) uk[t] = *reinterpret_cast<const f32x4 *>(rows->uk + 16 * t + q4);
                const float sn = rows->sn, total = rows->total;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    gk[t] = gk[t] * ss.inv;
#pragma unroll
                    for (int r = 0; r < 4; ++r) z[t][r] = fmaf(-gk[t][r], acc[t][r], __builtin_bit_cast(float, v[4 * t + r]));
                    acc[t] = f32x4{0, 0, 0, 0};
                }
                if (c + 1 < live) load_v(c + 1);
                const Scale sz = scale_of(channel_max(largest(z)));
                Terms<2> zs[2];
                stack(z[0], z[1], sz.f, zs[0]);
                stack(z[2], z[3], sz.f, zs[1]);
                const float back = sn * sz.inv;
#pragma unroll
                for (int P = 0; P < 2; ++P)
#pragma unroll
                    for (int t = 2 * P; t < 4; ++t) acc[t] = mma(ns[lower(t, P)], zs[P], acc[t]);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) z[t][r] = fmaf(acc[t][r], back, z[t][r]);      // Y
                    x.y[t][lane] = z[t];
                    z[t] = z[t] * uk[t];
                }
                const Scale su = scale_of(channel_max(largest(z)));
                Terms<2> us[2];
                stack(z[0], z[1], su.f, us[0]);
                stack(z[2], z[3], su.f, us[1]);
#pragma unroll
                for (int i = 0; i < SP / 16; ++i) {
                    f32x4 d = {0, 0, 0, 0};
#pragma unroll
                    for (int P = 0; P < 2; ++P) {
                        Terms<NI> a;
#pragma unroll
                        for (int e = 0; e < NI; ++e) a.f[e] = get_transposed<KS>(kn + e * 4 * KS * kOp, P, i >> 1, i & 1, lane);
                        d = mma(a, us[P], d);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) st[i][r] = fmaf(d[r], su.inv, st[i][r] * total);
                }
            }
            meet();
        }
        store_state<SP>(p.state_out + (nh * p.P + chc) * p.S, p.state_out && mine, p.S, lane, st);
    } else {
        T *yg = (T *)p.y + n * p.L * p.y_ld + (int64_t)h * p.P + chc;
        // Q and M of a chunk, fetched a chunk ahead
        struct Operands {
            Terms<NI> q[4 * KS], m[kTri];
            f32x4 gq[4], mq[4];
        } even, odd;
        auto step = [&](int c, Operands &next, const Operands &o) {
            if (NB == 1) {
                if (c < live) fetch_chunk(c);
                wait_vmcnt<0>();
                meet();
            } else if (c + 1 < live) {
                fetch_chunk(c + 1);
            }
            if (c < live) {
                const char *a = keys + c * keys_step + KEYS, *b = heads + c * head_step;
                const ChunkRows *rows = reinterpret_cast<const ChunkRows *>(b + kHeadRows);
#pragma unroll
                for (int f = 0; f < 4 * KS; ++f) get_terms(a + f * kOp, 4 * KS * kOp, lane, next.q[f]);
#pragma unroll
                for (int f = 0; f < kTri; ++f) get_terms(b + kHeadM + f * kOp, kTri * kOp, lane, next.m[f]);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    next.gq[t] = *reinterpret_cast<const f32x4 *>(rows->gq + 16 * t + q4);
                    next.mq[t] = *reinterpret_cast<const f32x4 *>(rows->mq + 16 * t + q4);
                }
            }
            if (c > 0) {
                const typename Shared::Exchange &x = sh.x[(c - 1) & 1][s_wave];
                f32x4 a1[4], a2[4], y[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a1[t] = a2[t] = f32x4{0, 0, 0, 0}, y[t] = x.y[t][lane];
                const float inv = x.inv[l16];
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    Terms<NI> b;
                    get_terms(x.s + s * kOp, KS * kOp, lane, b);
#pragma unroll
                    for (int t = 0; t < 4; ++t) a1[t] = mma(o.q[t * KS + s], b, a1[t]);
                }
                const Scale sy = scale_of(channel_max(largest(y)));
                Terms<NI> ys[2];
                stack(y[0], y[1], sy.f, ys[0]);
                stack(y[2], y[3], sy.f, ys[1]);
#pragma unroll
                for (int P = 0; P < 2; ++P)
#pragma unroll
                    for (int t = 2 * P; t < 4; ++t) a2[t] = mma(o.m[lower(t, P)], ys[P], a2[t]);
                const int64_t t0 = (int64_t)(c - 1) * kDQ;
                const LaneRows<T> rows((const T *)p.y + (int64_t)h * p.P, p.y_ld, n * p.L + t0, (int)(len - t0 < kDQ ? len - t0 : kDQ), p.P,
                                       ch, lane);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const f32x4 g1 = o.gq[t] * inv, g2 = o.mq[t] * sy.inv;
#pragma unroll
                    for (int r = 0; r < 4; ++r) rows.put(4 * t + r, fmaf(a1[t][r], g1[r], a2[t][r] * g2[r]));
                }
            }
            wait_vmcnt<0>();            // the next chunk's operands are there
            meet();
        };
        if (NB == 2 && live > 0) fetch_chunk(0);
        wait_vmcnt<0>();
        meet();
        for (int c = 0; c <= live; c += 2) {
            step(c, even, odd);
            if (c < live) step(c + 1, odd, even);
        }
        if (mine)
            for (int64_t t = len + (lane >> 4); t < p.L; t += 4) yg[t * p.y_ld] = (T)0.0f;
    }
}

}  // namespace convfwd
