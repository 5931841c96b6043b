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
// enters as the sum of three bf16 numbers, each the rounding of what the ones
// before it left, so that all 24 bits of it take part (with two terms for M and
// h, 16 bits, one y in a thousand was a bf16 neighbour of what fp32 gives; the
// third costs 3 to 8%).  fp32 calls run on the fp32 matrix instructions instead.
// States, sums and exponents are fp32; the running sums c_i are added in fp64 and
// used as differences, which are rounded to fp32 only then (c_i itself, up to some
// hundreds, would be off by 1e-5, and so would every decay; behind a token whose
// step clears the state it is thousands): two fp32 numbers stand for c_i.
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
    int nseg, seg, sub;         // segments of a sequence, chunks of a segment, segments of a forward workgroup
    int softplus, vec;
    int64_t ahead;              // workgroups of the state kernels that run ahead; the others run back
    float *seg_state[2], *seg_log[2];   // ahead and back: [unit][nseg][SP][64] (forward: [64][SP]), [unit][nseg]
    float *bound[2];            // [unit][K][SP][64]: the state and its gradient at every chunk's border
    // gradient
    const void *dy;
    const float *dstate_out;
    void *dx, *ddt, *db, *dc;
    float *dstate;
    int64_t dy_ld, dx_ld, ddt_ld, db_ld, dc_ld;
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
    // Row padding of the LDS tiles, elements: 32 bytes.  Rows are 128 or 256 bytes;
    // with 32 more, the 16 rows of a fragment and the 4 rows of a transposing read
    // take 4.0 clocks a wave instruction each (16 more: 8.0 and 4.0).
    static constexpr int PAD = 16;
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
// two values rounded to bf16 in one word, and taken off them
SEQ_DEV uint32_t take_pair(float &a, float &b)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
    a -= __builtin_bit_cast(float, w << 16);
    b -= __builtin_bit_cast(float, w & 0xffff0000u);
    return w;
}
template <int NS> SEQ_DEV void make_split(const float (&v)[8], Split<bf16_t, NS> &s)
{
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = take_pair(r[2 * e], r[2 * e + 1]);
        s.f[k] = __builtin_bit_cast(bf16x8, w);
    }
}
template <int NS> SEQ_DEV void make_split(const float (&v)[8], Split<float, NS> &s)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) s.f[0].v[e] = v[e];
}
// fp32 needs one term only
template <typename T, int NS> constexpr int terms() { return sizeof(T) == 4 ? 1 : NS; }

// The bf16 matrix unit rounds its sums down, by a few hundredths of a step on
// average: where they meet x, B or C of one sign it adds up over the tokens.
// The gradient takes half of its products of negated operands (`flip`: their
// sign bits) and negates the sums: ddt_bias of 2 x 2048 tokens is off by 2e-7 of
// itself instead of 1.4e-6, for 2 of 80 us.
SEQ_DEV bf16x8 flipped(bf16x8 f, uint32_t flip)
{
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4_t, f) ^ (u32x4_t)(flip));
}
SEQ_DEV Frag<float>::type flipped(const Frag<float>::type &f, uint32_t) { return f; }
template <typename T> SEQ_DEV uint32_t flip_of(bool odd) { return sizeof(T) == 2 && odd ? 0x80008000u : 0; }

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
            float a = v[0], b = v[1], c = v[2], d = v[3];
            const uint32_t lo = take_pair(a, b), hi = take_pair(c, d);
            v = f32x4{a, b, c, d};
            *reinterpret_cast<uint64_t *>(t + k * term_stride) = (uint64_t)hi << 32 | lo;
        }
    }
}

// ---- tiles -------------------------------------------------------------------
// ROWS x COLS of a matrix with `ld` elements from row to row, through THREADS
// threads' registers into LDS and back, by buffer accesses: a lane's offsets
// are the same for every chunk, and what lies outside `rows` x `cols` comes out
// as zeros, is never read (it may hold anything) and is not written, without a
// branch.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStream = 2;      // the non-temporal hint of a buffer access: outputs are not read back

template <typename T, int ROWS, int COLS, int THREADS = 256> struct Tile {
    static constexpr int VE = Frag<T>::VE;
    static constexpr int ALL = ROWS * COLS / VE;        // vectors of the tile
    static constexpr int NV = (ALL + THREADS - 1) / THREADS;
    static constexpr int LD = COLS + Frag<T>::PAD;
    static constexpr int CV = COLS / VE;
    static_assert(ALL % THREADS == 0 || ALL < THREADS, "whole vectors per thread");
    static SEQ_DEV bool mine() { return ALL >= THREADS || (int)threadIdx.x < ALL; }
    static constexpr uint32_t kOut = 0x80000000u;       // an offset past any buffer
    u32x4 v[NV];

    // the buffer that ends with the last valid element
    static SEQ_DEV __amdgpu_buffer_rsrc_t buffer(const T *g, int64_t ld, int rows, int cols)
    {
        const int bytes = rows > 0 ? (int)(((rows - 1) * ld + cols) * (int64_t)sizeof(T)) : 0;
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<T *>(g), 0, bytes, 0x00020000);
    }
    // A thread's k-th vector lies kStep rows behind its first, whose byte offset
    // and column are these.  opaque() keeps the others from being computed once
    // and held in registers.
    static constexpr int kStep = THREADS / CV;
    static SEQ_DEV int column() { return (int)threadIdx.x % CV * VE; }
    static SEQ_DEV uint32_t first(int64_t ld, int cols)
    {
        const int r = threadIdx.x / CV, c = column();
        return c < cols && mine() ? (uint32_t)(r * (int)ld + c) * (uint32_t)sizeof(T) : kOut;
    }
    static SEQ_DEV uint32_t opaque(uint32_t v)
    {
        asm volatile("" : "+v"(v));
        return v;
    }
    SEQ_DEV void load(const T *g, int64_t ld, int rows, int cols, bool vec)
    {
        const __amdgpu_buffer_rsrc_t buf = buffer(g, ld, rows, cols);
        const uint32_t step = (uint32_t)(kStep * (int)ld * (int)sizeof(T));
        uint32_t o = opaque(first(ld, cols));
        if (vec) {
#pragma unroll
            for (int k = 0; k < NV; ++k) v[k] = __builtin_amdgcn_raw_buffer_load_b128(buf, o + k * step, 0, 0);
        } else {
            const int left = (int)opaque(mine() ? cols - column() : 0);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int i = 0; i < VE; ++i)
                        v[k][i] = __builtin_amdgcn_raw_buffer_load_b32(buf, i < left ? o + i * 4 : kOut, 0, 0);
                } else {
#pragma unroll
                    for (int i = 0; i < VE; i += 2) {
                        const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(buf, i < left ? o + i * 2 : kOut, 0, 0);
                        const uint32_t hi =
                            __builtin_amdgcn_raw_buffer_load_b16(buf, i + 1 < left ? o + i * 2 + 2 : kOut, 0, 0);
                        v[k][i / 2] = (lo & 0xffffu) | (hi << 16);
                    }
                }
                o = opaque(o + step);
            }
        }
    }
    SEQ_DEV void store(T *lds) const
    {
        T *p = lds + threadIdx.x / CV * LD + column();
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (mine()) *reinterpret_cast<u32x4 *>(p + k * kStep * LD) = v[k];
    }
    // from LDS to memory, zeros in the rows from `live` on (what was computed there
    // is zero times a state, which need not be finite)
    static SEQ_DEV void write(const T *lds, T *g, int64_t ld, int live, int rows, int cols, bool vec)
    {
        Tile t;
        const int r = threadIdx.x / CV;
        const T *p = lds + r * LD + column();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            t.v[k] = u32x4{0, 0, 0, 0};
            if (mine() && r + k * kStep < live) t.v[k] = *reinterpret_cast<const u32x4 *>(p + k * kStep * LD);
        }
        t.put(g, ld, rows, cols, vec);
    }
    static SEQ_DEV void write_zeros(T *g, int64_t ld, int rows, int cols, bool vec)
    {
        Tile t;
#pragma unroll
        for (int k = 0; k < NV; ++k) t.v[k] = u32x4{0, 0, 0, 0};
        t.put(g, ld, rows, cols, vec);
    }
    SEQ_DEV void put(T *g, int64_t ld, int rows, int cols, bool vec) const
    {
        const __amdgpu_buffer_rsrc_t buf = buffer(g, ld, rows, cols);
        const uint32_t step = (uint32_t)(kStep * (int)ld * (int)sizeof(T));
        uint32_t o = opaque(first(ld, cols));
        if (vec) {
#pragma unroll
            for (int k = 0; k < NV; ++k) __builtin_amdgcn_raw_buffer_store_b128(v[k], buf, o + k * step, 0, kStream);
        } else {
            const int left = (int)opaque(mine() ? cols - column() : 0);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const uint32_t at = i < left ? o + i * (uint32_t)sizeof(T) : kOut;
                    if constexpr (sizeof(T) == 4)
                        __builtin_amdgcn_raw_buffer_store_b32(v[k][i], buf, at, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v[k][i / 2] >> (i & 1) * 16), buf, at, 0, 0);
                }
                o = opaque(o + step);
            }
        }
    }
};

// The compiler, left alone, reads one fragment from LDS, waits for it and
// multiplies, and each wait is a round trip. The kernels read fragments in
// groups, a group ahead of the products, and keep the order with this.
SEQ_DEV void in_order() { __builtin_amdgcn_sched_barrier(0); }

// a value the compiler cannot know to be the same as before
SEQ_DEV int fresh_vector(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}
SEQ_DEV int fresh_scalar(int v)
{
    asm volatile("" : "+s"(v));
    return v;
}

SEQ_DEV int64_t fresh_scalar(int64_t v)
{
    asm volatile("" : "+s"(v));
    return v;
}

// the wave's number in the workgroup, known to be the same in all its lanes
SEQ_DEV int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// ---- wave helpers --------------------------------------------------------------
// One step of a sum over lanes: v of the lane that DPP control `ctrl` names, or
// 0 where it names none or the row is masked out.
template <int CTRL, int ROWS> SEQ_DEV float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS> SEQ_DEV double dpp(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)b, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// inclusive sums over the 64 lanes: shifts within rows of 16, then row 0's sum
// into row 1 and 2's into 3, then the first half's into the second
template <typename V> SEQ_DEV V wave_prefix(V v)
{
    v += dpp<0x111, 0xf>(v);
    v += dpp<0x112, 0xf>(v);
    v += dpp<0x114, 0xf>(v);
    v += dpp<0x118, 0xf>(v);
    v += dpp<0x142, 0xa>(v);
    v += dpp<0x143, 0xc>(v);
    return v;
}
SEQ_DEV float wave_last(float v) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63)); }
SEQ_DEV double wave_last(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)b, 63), hi = __builtin_amdgcn_readlane((int)(b >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
SEQ_DEV float wave_sum(float v) { return wave_last(wave_prefix(v)); }
// The sums of v[0..3] over the 16 lanes of a row, v[r]'s in the lanes 4r..4r+3:
// two exchanges that halve the values, then two within the four lanes.
template <typename V = float> SEQ_DEV V row_sum4(f32x4 v, int lane)
{
    const bool b3 = lane & 8, b2 = lane & 4;
    const V a = (V)(b3 ? v[2] : v[0]) + (V)dpp<0x128, 0xf>(b3 ? v[0] : v[2]);   // 8 lanes on
    const V b = (V)(b3 ? v[3] : v[1]) + (V)dpp<0x128, 0xf>(b3 ? v[1] : v[3]);
    V s = (b2 ? b : a) + dpp<0x141, 0xf>(b2 ? a : b);                           // mirrored in 8 lanes
    s += dpp<0xb1, 0xf>(s);
    s += dpp<0x4e, 0xf>(s);
    return s;
}

// Token `lane` of a chunk: the step size dt (0 behind the sequence) and the
// running sum of log2 of the decays, in fp64.  A decay under 2^-1024 counts as
// that, zero in fp32 like whatever it is a factor of: a step that clears the
// state may be any number and leaves the sums their digits.
SEQ_DEV void chunk_decay(float raw, bool live, float a, int softplus_on, float &dt, double &cum)
{
    dt = live ? (softplus_on ? softplus(raw) : raw) : 0.0f;
    const double decay = (double)a * (double)dt * 1.4426950408889634074;
    cum = wave_prefix(decay < -1024.0 ? -1024.0 : decay);
}


// ---- states at the chunks' borders, and at the segments' ------------------------
// (fp32 calls and bf16 rows that are no whole vectors; the others are in
// scan_dma.h.)  The products with B are a quarter of the forward's; what a chunk
// costs beside them is its way through registers into LDS and the decays' chain,
// so four chunks' decays are done at once, one by each wave.  16384 tokens x 64
// heads in bf16: 78 us against scan_dma.h's 62-70; fp32, 777 tokens x 12 sequences
// and heads of 40 channels x 24 states: 6.0 us, the launch and three chunks' loads.
// One workgroup: 64 channels of a head, one segment of chunks, wave w the
// channels 16w..16w+15 and all of the state (results: rows channels, columns
// states).  Run back (REV) from the last chunk to the first it takes dy, C and
// weights e^{c_i} instead of x, B and e^{c_Q - c_j} dt_j: the state's gradient.
// STORE leaves the state at every chunk's near border in `bound` and starts
// from the segment's own start; without it the segment starts from zero and
// leaves its last state and the logarithm of its decay.
template <typename T, int SP> struct StateShared {
    static constexpr int Q = Frag<T>::Q;
    __align__(16) T x[Q * Tile<T, Q, kPB>::LD];
    __align__(16) T b[Q * Tile<T, Q, SP>::LD];
    __align__(16) float w[4][Q];        // the weights of four chunks in a row
    float tot[4];
};

// The state that a segment starts from: what came before the sequence, then the
// states that the segments before left from zero, each decayed by those between.
// get(s, t) is the lane's four values of result t in a segment's state s; the
// loads of several segments are under way together.
template <int SP, bool REV, typename F>
SEQ_DEV void join_segments(const ScanParams &p, int64_t unit, int seg, f32x4 (&acc)[SP / 16], F &&get)
{
    constexpr int NT = SP / 16, AT = 24 / NT;
    const float *s = p.seg_state[REV] + unit * p.nseg * (SP * kPB), *lg = p.seg_log[REV] + unit * p.nseg;
    const int count = REV ? p.nseg - 1 - seg : seg;
    for (int k0 = 0; k0 < count; k0 += AT) {
        f32x4 v[AT][NT];
        float dec[AT];
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            const int k = min(k0 + i, count - 1), from = REV ? p.nseg - 1 - k : k;
            dec[i] = lg[from];
#pragma unroll
            for (int t = 0; t < NT; ++t) v[i][t] = get(s + (int64_t)from * (SP * kPB), t);
        }
        in_order();
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            if (k0 + i < count) {
                const float d = exp2_fast(dec[i]);
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t] = acc[t] * d + v[i][t];
            }
        }
    }
}

// ... as rows (channels ch .., four) x columns (states 16 t + lane % 16)
template <int SP, bool REV>
SEQ_DEV void start_states(const ScanParams &p, int64_t unit, int seg, int ch, int pcols, int lane, f32x4 (&acc)[SP / 16])
{
    constexpr int NT = SP / 16;
    const float *s = REV ? p.dstate_out : p.state;
    if (s) {
        s += (unit / p.NPB * p.P + unit % p.NPB * kPB) * p.S;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (ch + r < pcols && t * 16 + (lane & 15) < p.S) acc[t][r] = s[(int64_t)(ch + r) * p.S + t * 16 + (lane & 15)];
    }
    join_segments<SP, REV>(p, unit, seg, acc, [&](const float *v, int t) __attribute__((always_inline)) {
        return *reinterpret_cast<const f32x4 *>(v + (t * 16 + (lane & 15)) * kPB + ch);
    });
}

// What a segment leaves from zero, in the order in which the next kernel takes
// four neighbours at once: channels for the gradient, states for the forward.
template <int SP>
SEQ_DEV void leave_segment(const ScanParams &p, float *seg_state, float *seg_log, int64_t unit, int seg, int ch, int lane,
                           float log_dec, const f32x4 (&acc)[SP / 16])
{
    float *s = seg_state + (unit * p.nseg + seg) * (SP * kPB);
#pragma unroll
    for (int t = 0; t < SP / 16; ++t) {
        const int state = t * 16 + (lane & 15);
        if (p.y) {
#pragma unroll
            for (int r = 0; r < 4; ++r) s[(ch + r) * SP + state] = acc[t][r];
        } else {
            *reinterpret_cast<f32x4 *>(s + state * kPB + ch) = acc[t];
        }
    }
    if (threadIdx.x == 0) seg_log[unit * p.nseg + seg] = log_dec;
}

template <typename T, int SP, bool REV, bool STORE>
SEQ_DEV void scan_states(const ScanParams &p, int64_t block, StateShared<T, SP> &sh)
{
    constexpr int Q = Frag<T>::Q, NT = SP / 16, NS = terms<T, 3>();
    typedef Tile<T, Q, kPB> XT;
    typedef Tile<T, Q, SP> BT;
    T *sX = sh.x, *sB = sh.b;
    float (*sW)[Q] = sh.w, *sTot = sh.tot;
    float *seg_state = p.seg_state[REV], *seg_log = p.seg_log[REV];
    const int lane = threadIdx.x & 63, w = wave_id(), q = lane >> 4;
    const int nseg = STORE ? p.nseg : p.nseg - 1;
    const int64_t unit = block / nseg;
    const int s0 = (int)(block - unit * nseg);
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
    if (STORE) start_states<SP, REV>(p, unit, seg, ch, pcols, lane, acc);

    XT xt;
    BT bt;
    float raw = 0.0f, log_dec = 0.0f;
    auto fetch = [&](int c) __attribute__((always_inline)) {
        const int64_t t0 = (int64_t)c * Q;
        const int rows = (int)min((int64_t)Q, len - t0);
        xt.load(xg + t0 * x_ld, x_ld, rows, pcols, p.vec);
        bt.load(bg + t0 * b_ld, b_ld, rows, p.S, p.vec);
    };
    // The chunks' decays are a long chain of scalar work: each wave does one of
    // four chunks in a row, all at the same time, with its dt fetched ahead.
    auto chunk_of = [&](int k) __attribute__((always_inline)) { return REV ? c_live - 1 - (k - c_lo) : k; };
    auto fetch_dt = [&](int k) __attribute__((always_inline)) {
        const int64_t t = (int64_t)chunk_of(k) * Q + lane;
        raw = k < c_live && lane < Q && t < len ? (float)dg[t * p.dt_ld] + bias : 0.0f;
    };
    if (c_lo < c_live) {
        fetch_dt(c_lo + w);
        fetch(chunk_of(c_lo));
    }
    for (int k = c_lo; k < c_live; ++k) {
        const int c = chunk_of(k), slot = (k - c_lo) & 3;
        __syncthreads();
        xt.store(sX);
        bt.store(sB);
        if (slot == 0) {
            float dt;
            double cum;
            chunk_decay(raw, k + w < c_live && lane < Q && (int64_t)chunk_of(k + w) * Q + lane < len, a, p.softplus, dt, cum);
            const double tot = wave_last(cum);
            if (lane < Q) sW[w][lane] = REV ? exp2_fast((float)cum) : exp2_fast((float)(tot - cum)) * dt;
            if (lane == 0) sTot[w] = (float)tot;
            fetch_dt(k + 4 + w);
        }
        __syncthreads();
        if (k + 1 < c_live) fetch(REV ? c - 1 : c + 1);
        if (STORE) {
            float *s = p.bound[REV] + (unit * p.K + c) * (SP * kPB);
#pragma unroll
            for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4 *>(s + (t * 16 + (lane & 15)) * kPB + ch) = acc[t];
        }
        const float tot = sTot[slot], dec = exp2_fast(tot);
        log_dec += tot;
        if (busy) {
            constexpr int KS = Q / 32;
            typename Frag<T>::type xf[KS], bf[KS][NT];
            f32x4 wt[KS][2];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                xf[ks] = read_cols(sX, XT::LD, ks * 32, w * 16, lane);
                wt[ks][0] = *reinterpret_cast<const f32x4 *>(&sW[slot][ks * 32 + q * 8]);
                wt[ks][1] = *reinterpret_cast<const f32x4 *>(&sW[slot][ks * 32 + q * 8 + 4]);
            }
            auto read_b = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
                for (int t = 0; t < NT; ++t) bf[ks][t] = read_cols(sB, BT::LD, ks * 32, t * 16, lane);
            };
            read_b(0);
            in_order();
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] *= dec;
            Split<T, NS> xs[KS];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = frag_get(xf[ks], e) * wt[ks][e / 4][e & 3];
                make_split(v, xs[ks]);
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if (ks + 1 < KS) read_b(ks + 1);
                in_order();
#pragma unroll
                for (int m = 0; m < NS; ++m)
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[t] = mma(xs[ks].f[m], bf[ks][t], acc[t]);
            }
        }
    }
    if (!STORE) {
        leave_segment<SP>(p, seg_state, seg_log, unit, seg, ch, lane, log_dec, acc);
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

template <typename T, int SP, bool STORE> __global__ void __launch_bounds__(256) scan_state_kernel(ScanParams p)
{
    __shared__ StateShared<T, SP> sh;
    if (blockIdx.x < p.ahead) scan_states<T, SP, false, STORE>(p, blockIdx.x, sh);
    else scan_states<T, SP, true, STORE>(p, blockIdx.x - p.ahead, sh);
}

// Lower-triangle tile t of the chunk's scores: row it, column jt <= it
SEQ_DEV void tri_tile(int t, int &it, int &jt)
{
    it = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
    jt = t - it * (it + 1) / 2;
}

// ---- forward -------------------------------------------------------------------
// (fp32 calls and bf16 rows that are no whole vectors; the others are in
// scan_dma.h.)
// One workgroup: 64 channels of a head, one segment of chunks; wave w keeps the
// state of channels 16w..16w+15 in registers (results: rows states, columns
// channels, which makes them the operand of h_0 C as they stand).  The chunk's
// scores are computed once, their 16x16 tiles dealt to the waves, and pass
// through LDS as M.  The workgroup waits at four barriers a chunk; two of them
// share a compute unit (251 registers, 80 KB of LDS).  16384 tokens x 64 heads in
// bf16 take 300 us with this kernel and the pass before it, 226 with scan_dma.h's;
// fp32, 777 tokens x 12 heads of 40 x 24: 13 us, of which the join of up to 9
// segments is half.
template <typename T, int SP> __global__ void __launch_bounds__(256, 2) scan_fwd_kernel(ScanParams p)
{
    constexpr int Q = Frag<T>::Q, NT = SP / 16, NI = Q / 16, TRI = NI * (NI + 1) / 2, TPW = (TRI + 3) / 4;
    constexpr int NS = terms<T, 3>(), MLD = Q + Frag<T>::PAD;
    typedef Tile<T, Q, kPB> XT;
    typedef Tile<T, Q, SP> BT;
    typedef typename Frag<T>::type frag;
    __shared__ __align__(16) T sX[Q * XT::LD];
    __shared__ __align__(16) T sB[Q * BT::LD];
    __shared__ __align__(16) T sC[Q * BT::LD];
    __shared__ __align__(16) T sM[NS * Q * MLD];
    // of four chunks: c_i, its low part, dt, e^{c_Q - c_j} dt_j (e^{c_i} besides would leave room for one workgroup only)
    __shared__ __align__(16) float sCum[4][Q], sLow[4][Q], sDt[4][Q], sW[4][Q];
    const int lane = threadIdx.x & 63, w = wave_id(), q = lane >> 4;
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
    if (p.state && col < pcols) {
        const float *s = p.state + (nh * p.P + pb * kPB + col) * p.S;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (t * 16 + q * 4 + r < p.S) st[t][r] = s[t * 16 + q * 4 + r];
    }
    join_segments<SP, false>(p, unit, seg, st, [&](const float *v, int t) __attribute__((always_inline)) {
        return *reinterpret_cast<const f32x4 *>(v + col * SP + t * 16 + q * 4);
    });
    // the tiles of M above the diagonal that a reduction over 32 tokens meets
    for (int e = threadIdx.x; e < NS * Q * MLD; e += 256) sM[e] = (T)0.0f;

    XT xt;
    BT bt, ct;
    float raw = 0.0f;
    auto fetch = [&](int c) __attribute__((always_inline)) {
        const int64_t t0 = (int64_t)c * Q;
        const int rows = (int)min((int64_t)Q, len - t0);
        xt.load(xg + t0 * p.x_ld, p.x_ld, rows, pcols, p.vec);
        bt.load(bg + t0 * p.b_ld, p.b_ld, rows, p.S, p.vec);
        ct.load(cg + t0 * p.c_ld, p.c_ld, rows, p.S, p.vec);
    };
    auto fetch_dt = [&](int c) __attribute__((always_inline)) {      // as in scan_state_kernel
        const int64_t t = (int64_t)c * Q + lane;
        raw = c < c_live && lane < Q && t < len ? (float)dg[t * p.dt_ld] + bias : 0.0f;
    };
    if (c_lo < c_live) {
        fetch_dt(c_lo + w);
        fetch(c_lo);
    }
    for (int c = c_lo; c < c_live; ++c) {
        const int64_t t0 = (int64_t)c * Q;
        const int slot = (c - c_lo) & 3;
        const float *cum_ = sCum[slot], *low_ = sLow[slot], *dt_ = sDt[slot], *w_ = sW[slot];
        __syncthreads();
        xt.store(sX);
        bt.store(sB);
        ct.store(sC);
        if (slot == 0) {
            float dt;
            double cum;
            chunk_decay(raw, c + w < c_live && lane < Q && t0 + w * Q + lane < len, a, p.softplus, dt, cum);
            const double tot = wave_last(cum);
            if (lane < Q) {
                sDt[w][lane] = dt;
                sCum[w][lane] = (float)cum;
                sLow[w][lane] = (float)(cum - (double)(float)cum);
                sW[w][lane] = exp2_fast((float)(tot - cum)) * dt;
            }
            fetch_dt(c + 4 + w);
        }
        __syncthreads();
        if (c + 1 < c_live) fetch(c + 1);
        // M, tile by tile: rows j, column i in a lane, so four neighbours of a row of M
        {
            constexpr int KN = SP / 32;
#pragma unroll
            for (int k = 0; k < TPW; ++k) {
                if (w + 4 * k < TRI) {
                    int it, jt;
                    tri_tile(w + 4 * k, it, jt);
                    frag bf[KN], cf[KN];
#pragma unroll
                    for (int ks = 0; ks < KN; ++ks) {
                        bf[ks] = read_rows(sB, BT::LD, jt * 16, ks * 32, lane);
                        cf[ks] = read_rows(sC, BT::LD, it * 16, ks * 32, lane);
                    }
                    const int i = it * 16 + (lane & 15), j = jt * 16 + q * 4;
                    const f32x4 dj = *reinterpret_cast<const f32x4 *>(dt_ + j);
                    const f32x4 ex = (cum_[i] - *reinterpret_cast<const f32x4 *>(cum_ + j)) +
                                     (low_[i] - *reinterpret_cast<const f32x4 *>(low_ + j));
                    in_order();
                    f32x4 s = {0, 0, 0, 0};
#pragma unroll
                    for (int ks = 0; ks < KN; ++ks) s = mma(bf[ks], cf[ks], s);
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[r] = i >= j + r ? s[r] * exp2_fast(ex[r]) * dj[r] : 0.0f;
                    write_split4<NS>(sM + i * MLD + j, Q * MLD, s);
                }
            }
        }
        __syncthreads();
        if (busy) {
            constexpr int KQ = Q / 32, KN = SP / 32;
            frag xf[KQ], cf[2][NI], mf[NI][NS], bf[NT];
            f32x4 y[NI];
            auto read_c = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
                for (int it = 0; it < NI; ++it) cf[ks & 1][it] = read_rows_stacked(sC, BT::LD, it * 16, ks * 32, lane);
            };
            auto read_m = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
                for (int it = 2 * ks; it < NI; ++it)
#pragma unroll
                    for (int m = 0; m < NS; ++m) mf[it][m] = read_rows(sM + m * Q * MLD, MLD, it * 16, ks * 32, lane);
            };
            auto read_b = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
                for (int t = 0; t < NT; ++t) bf[t] = read_cols(sB, BT::LD, ks * 32, t * 16, lane);
            };
#pragma unroll
            for (int it = 0; it < NI; ++it) y[it] = f32x4{0, 0, 0, 0};
            read_c(0);
            // e^{c_i} h_0 C_i, the next fragments on their way
#pragma unroll
            for (int ks = 0; ks < KN; ++ks) {
                if (ks + 1 < KN) {
                    read_c(ks + 1);
                } else {
#pragma unroll
                    for (int k = 0; k < KQ; ++k) xf[k] = read_cols(sX, XT::LD, k * 32, w * 16, lane);
                    read_m(0);
                }
                in_order();
                float v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = st[2 * ks][e], v[4 + e] = st[2 * ks + 1][e];
                Split<T, NS> hs;
                make_split(v, hs);
#pragma unroll
                for (int m = 0; m < NS; ++m)
#pragma unroll
                    for (int it = 0; it < NI; ++it) y[it] = mma(cf[ks & 1][it], hs.f[m], y[it]);
                in_order();
            }
#pragma unroll
            for (int it = 0; it < NI; ++it)
#pragma unroll
                for (int r = 0; r < 4; ++r) y[it][r] *= exp2_fast(cum_[it * 16 + q * 4 + r]);
            const float dec = exp2_fast(cum_[Q - 1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) st[t] *= dec;
            T xr[NI][4];
#pragma unroll
            for (int ks = 0; ks < KQ; ++ks) {
                in_order();
                read_b(ks);
                const f32x4 w0 = *reinterpret_cast<const f32x4 *>(w_ + ks * 32 + q * 8);
                const f32x4 w1 = *reinterpret_cast<const f32x4 *>(w_ + ks * 32 + q * 8 + 4);
                in_order();
#pragma unroll
                for (int m = 0; m < NS; ++m)
#pragma unroll
                    for (int it = 2 * ks; it < NI; ++it) y[it] = mma(mf[it][m], xf[ks], y[it]);
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = frag_get(xf[ks], e) * (e < 4 ? w0[e & 3] : w1[e & 3]);
                Split<T, NS> xs;
                make_split(v, xs);
                in_order();
                if (ks + 1 < KQ) {
                    read_m(ks + 1);
                } else {
#pragma unroll
                    for (int it = 0; it < NI; ++it)
#pragma unroll
                        for (int r = 0; r < 4; ++r) xr[it][r] = sX[(it * 16 + q * 4 + r) * XT::LD + col];
                }
                in_order();
#pragma unroll
                for (int m = 0; m < NS; ++m)
#pragma unroll
                    for (int t = 0; t < NT; ++t) st[t] = mma(bf[t], xs.f[m], st[t]);
            }
            // y in place of this wave's own columns of x
#pragma unroll
            for (int it = 0; it < NI; ++it)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sX[(it * 16 + q * 4 + r) * XT::LD + col] = (T)fmaf(skip, (float)xr[it][r], y[it][r]);
        }
        __syncthreads();
        XT::write(sX, yg + t0 * p.y_ld, p.y_ld, (int)min((int64_t)Q, len - t0), (int)min((int64_t)Q, p.L - t0), pcols, p.vec);
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
// One workgroup of eight waves: one chunk of one group, a slice of the group's
// heads (in blocks of 64 channels) one after the other.  C . B is the same for
// all of them and stays in registers, and so do the sums of dS over the heads,
// from which dB and dC get their parts inside the chunk by one product each at
// the end.  The waves share dP's 16x16 tiles as the forward shares its scores;
// dB and dC go by states (and tokens, where there are fewer than 8 x 16 states),
// dx by channels and halves of the tokens.  The states at the chunk's borders and
// their gradients come from memory, where the two runs of the state kernel left
// them.  While a head is computed the next one's x, dy and states are on their
// way into registers, wave 6 does its decays, and wave 7 turns the sums that the
// head before left in LDS into ddt and its parts of dA, ddt_bias and dD.
// 2 x 2048 tokens, 32 heads of 64 x 128 in bf16: 83 us, 10 a head and chunk for 32
// + 32 KB of states at its borders (1.6 TB/s); the products are 5 us of them, the
// other vector instructions (splits, decays, sums over lanes) 30, and the loads of
// the next states, which 256 registers leave no room to start earlier, most of the
// rest.  Four waves of 512 registers instead: 138 where 87 was the time; the sums
// over lanes one value at a time: 100; the tensors' addresses kept over the heads
// instead of taken anew: 82 for 78.
template <typename T, int SP> struct BwdShared {
    static constexpr int Q = Frag<T>::Q, NI = Q / 16, NS = terms<T, 3>();
    static constexpr int XLD = kPB + Frag<T>::PAD, BLD = SP + Frag<T>::PAD, MLD = Q + Frag<T>::PAD;
    static constexpr int ULD = kPB + 16 / (int)sizeof(T);       // few row fragments are read from u: half the padding
    __align__(16) T x[Q * XLD], y[Q * XLD];     // x and dy
    __align__(16) T b[Q * BLD], c[Q * BLD];
    __align__(16) T m[NS * Q * MLD];            // [term][j][i]
    __align__(16) T u[NS * SP * ULD];           // [term][state][channel]
    __align__(16) float dt[2][Q], cum[2][Q], low[2][Q], w[2][Q], e[2][Q], raw[2][Q];   // w: e^{c_Q - c_j}
    double row[2][NI][Q], col[2][NI][Q];        // of W: see finish()
    float cd[2][8][Q], xd[4][Q], xi[4][Q], dot[2][8], dd[2][8];
    double pairs[64];                           // wave 7's, from channel block to channel block of a head
    float sums[5][64];
};

template <typename T, int SP> __global__ void __launch_bounds__(512) scan_bwd_kernel(ScanParams p)
{
    typedef BwdShared<T, SP> Sh;
    constexpr int Q = Sh::Q, NI = Sh::NI, NS = Sh::NS, XLD = Sh::XLD, BLD = Sh::BLD, MLD = Sh::MLD, ULD = Sh::ULD;
    constexpr int NT = SP / 16, TRI = NI * (NI + 1) / 2, TW = 6, TPW = (TRI + TW - 1) / TW;    // waves 6 and 7 have other work
    constexpr int WN = NT, WI = 8 / WN, ITW = NI / WI > 0 ? NI / WI : 1, JW = NI / 2;
    typedef Tile<T, Q, kPB, 512> XT;
    typedef Tile<T, Q, SP, 512> BT;
    typedef typename Frag<T>::type frag;
    __shared__ Sh sh;
    const int lane = threadIdx.x & 63, w = wave_id(), q = lane >> 4, l16 = lane & 15;
    const int slice = (int)(blockIdx.x % p.slices);
    const int64_t ng = blockIdx.x / p.slices;
    const int g = (int)(ng % p.G);
    const int64_t nc = ng / p.G, n_ = nc / p.K, n = n_;
    const int c = (int)(nc - n * p.K), hpg = p.H / p.G;
    const int h_lo = slice * p.heads_per_slice, h_hi = min(hpg, h_lo + p.heads_per_slice);
    const int blocks = (h_hi - h_lo) * p.NPB;           // channel blocks of the slice's heads
    const int64_t len = seq_len(p.lengths, n, p.L), t0 = (int64_t)c * Q;
    const int rows = (int)max((int64_t)0, min((int64_t)Q, len - t0)), all_rows = (int)min((int64_t)Q, p.L - t0);
    const int64_t base_ = n * p.L + t0;       // the chunk's first row: taken anew where used, or every tensor's
                                              // address is computed once and kept
    const int64_t NK = (int64_t)p.N * p.K;
    const int nt = w % WN, it0 = w / WN * ITW;          // dB and dC: states 16 nt .., tokens 16 it0 ..
    const bool on = it0 < NI;

    XT xt, yt;
    float h0[16], u[16];        // state 16 nt + lane % 16, channels 32 ks + 8q + e at 8 ks + e
    auto head_of = [&](int k) __attribute__((always_inline)) { return g * hpg + h_lo + k / p.NPB; };
    auto fetch = [&](int k) __attribute__((always_inline)) {
        const int h = head_of(k), pb = k % p.NPB, pcols = min(kPB, p.P - pb * kPB);
        const int64_t xo = (int64_t)h * p.P + pb * kPB, base = fresh_scalar(base_);
        xt.load((const T *)p.x + base * p.x_ld + xo, p.x_ld, rows, pcols, p.vec);
        yt.load((const T *)p.dy + base * p.dy_ld + xo, p.dy_ld, rows, pcols, p.vec);
    };
    auto fetch_states = [&](int k) __attribute__((always_inline)) {
        const int h = head_of(k), pb = k % p.NPB;
        const int64_t n = fresh_scalar(n_);
        const int64_t o = (((n * p.H + h) * p.NPB + pb) * p.K + c) * (SP * kPB) + (nt * 16 + l16) * kPB + q * 8;
        // behind the sequence x, dy and dt are zeros: any finite state will do
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
            if (rows > 0) {
                a = *reinterpret_cast<const f32x4 *>(p.bound[0] + o + (i >> 1) * 32 + (i & 1) * 4);
                b = *reinterpret_cast<const f32x4 *>(p.bound[1] + o + (i >> 1) * 32 + (i & 1) * 4);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) h0[i * 4 + r] = a[r], u[i * 4 + r] = b[r];
        }
    };
    float raw = 0.0f;       // wave 6: of the head that comes next
    auto fetch_dt = [&](int k) __attribute__((always_inline)) {
        const int h = head_of(k);
        const int64_t base = fresh_scalar(base_);
        raw = lane < rows ? (float)((const T *)p.dt)[(base + lane) * p.dt_ld + h] + (p.dt_bias ? p.dt_bias[h] : 0.0f) : 0.0f;
    };
    auto decays = [&](int k) __attribute__((always_inline)) {
        const int h = head_of(k), to = (k / p.NPB) & 1;
        float dt;
        double cum;
        chunk_decay(raw, lane < rows, p.a[h], p.softplus, dt, cum);
        const double tot = wave_last(cum);
        if (lane < Q) {
            sh.raw[to][lane] = raw;
            sh.dt[to][lane] = dt;
            sh.cum[to][lane] = (float)cum;
            sh.low[to][lane] = (float)(cum - (double)(float)cum);
            sh.w[to][lane] = exp2_fast((float)(tot - cum));
            sh.e[to][lane] = exp2_fast((float)cum);
        }
    };
    // Wave 7, per token: the sums of a head over its channel blocks (in LDS from
    // block to block: as registers they would be everyone's), then what follows.
    // A pair i > j of W enters the sum over the pairs around each token as row i
    // less column j, so what a rounding takes from one of the two is left in every
    // token's sum: rows and columns are added in fp64, where the pair's fp32 value
    // cancels.  In fp32 ddt_bias was off by 1.0e-6 of itself, now by 2e-7 (the plain
    // products in fp32, summed in fp64: 4e-7), at the same time.
    auto finish = [&](int k) __attribute__((always_inline)) {
        const int at = k & 1, d = (k / p.NPB) & 1;
        double pairs = 0.0;
        float cd = 0.0f, ee = 0.0f, ei = 0.0f, dot = 0.0f, dd = 0.0f;
        if (k % p.NPB != 0) {
            pairs = sh.pairs[lane], cd = sh.sums[0][lane], ee = sh.sums[1][lane];
            ei = sh.sums[2][lane], dot = sh.sums[3][lane], dd = sh.sums[4][lane];
        }
        if (lane < Q) {
#pragma unroll
            for (int t = 0; t < NI; ++t) pairs += sh.row[at][t][lane] - sh.col[at][t][lane];
#pragma unroll
            for (int t = 0; t < WN; ++t) cd += sh.cd[at][t][lane];
#pragma unroll
            for (int t = 0; t < 4; ++t) ee += sh.xd[t][lane], ei += sh.xi[t][lane];
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) dot += sh.dot[at][t], dd += sh.dd[at][t];
        if (k % p.NPB != p.NPB - 1) {
            sh.pairs[lane] = pairs, sh.sums[0][lane] = cd, sh.sums[1][lane] = ee;
            sh.sums[2][lane] = ei, sh.sums[3][lane] = dot, sh.sums[4][lane] = dd;
            return;
        }
        const int h = head_of(k);
        const int64_t base = fresh_scalar(base_);
        const float dt = lane < Q ? sh.dt[d][lane] : 0.0f, raw = lane < Q ? sh.raw[d][lane] : 0.0f, dec = sh.e[d][Q - 1];
        const double before = (double)dt * ei, behind = pairs + cd;
        const double b1 = wave_prefix(before), b2 = wave_prefix(behind);
        float dl = (float)((b1 - before) + (wave_last(b2) - b2 + behind) + (double)(dec * dot));
        // every term has the token's decay as a factor; where that is zero, what the
        // sums leave is a rounding, and dt, which made it zero, may be any number
        if (p.a[h] * dt * kLog2e < -150.0f) dl = 0.0f;
        float draw = fmaf(p.a[h], dl, ee);
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
    };

    f32x4 sc[TPW], ds[TPW], dB[ITW], dC[ITW];
#pragma unroll
    for (int k = 0; k < TPW; ++k) sc[k] = ds[k] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < ITW; ++k) dB[k] = dC[k] = f32x4{0, 0, 0, 0};
    {
        BT bt, ct;
        bt.load((const T *)p.b + base_ * p.b_ld + (int64_t)g * p.S, p.b_ld, rows, p.S, p.vec);
        ct.load((const T *)p.c + base_ * p.c_ld + (int64_t)g * p.S, p.c_ld, rows, p.S, p.vec);
        fetch(0);
        fetch_states(0);
        bt.store(sh.b);
        ct.store(sh.c);
        // what is never written: M above its diagonal tiles, the same of the sums
        for (int e = threadIdx.x; e < NS * Q * MLD; e += 512) sh.m[e] = (T)0.0f;
        for (int e = threadIdx.x; e < 2 * NI * Q; e += 512) sh.row[0][0][e] = sh.col[0][0][e] = 0.0;
        if (w == 6) {
            fetch_dt(0);
            decays(0);
        }
    }
    __syncthreads();
    // scores: rows i, column j in a lane
#pragma unroll
    for (int k = 0; k < TPW; ++k) {
        const int t = w + TW * k;
        if (w < TW && t < TRI) {
            int it, jt;
            tri_tile(t, it, jt);
#pragma unroll
            for (int ks = 0; ks < SP / 32; ++ks)
                sc[k] = mma(read_rows(sh.c, BLD, it * 16, ks * 32, lane), read_rows(sh.b, BLD, jt * 16, ks * 32, lane), sc[k]);
        }
    }
    const int lane_ = lane, w_ = w;
    for (int k = 0; k < blocks; ++k) {
        // Addresses and masks follow from these two; taken anew each time they are
        // computed where they are used, or the compiler computes all of them ahead
        // of the loop and keeps them in memory.
        const int lane = fresh_vector(lane_), w = fresh_scalar(w_), q = lane >> 4, l16 = lane & 15;
        const int nt = w % WN, it0 = w / WN * ITW;
        const int pt = w & 3, jt0 = (w >> 2) * JW;      // dx: channels 16 pt .., tokens 16 jt0 ..
        const bool on = it0 < NI;
        const int at = k & 1, d = (k / p.NPB) & 1, h = head_of(k), pb = k % p.NPB, pcols = min(kPB, p.P - pb * kPB);
        const float skip = p.d ? p.d[h] : 0.0f;
        const float *s_cum = sh.cum[d], *s_low = sh.low[d], *s_dt = sh.dt[d], *s_w = sh.w[d], *s_e = sh.e[d];
        __syncthreads();        // all waves are done with the block before
        xt.store(sh.x);
        yt.store(sh.y);
        if (it0 == 0) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Split<T, NS> us;
                make_split(reinterpret_cast<const float (&)[8]>(u[ks * 8]), us);
#pragma unroll
                for (int m = 0; m < NS; ++m)
                    *reinterpret_cast<frag *>(sh.u + m * SP * ULD + (nt * 16 + l16) * ULD + ks * 32 + q * 8) = us.f[m];
            }
        }
        __syncthreads();
        if (k + 1 < blocks) {
            if (w == 6 && (k + 1) % p.NPB == 0) fetch_dt(k + 1);
        }
        // dP, M and dS, tile by tile; M goes to LDS transposed (rows j)
        float diag = 0.0f;
#pragma unroll
        for (int t8 = 0; t8 < TPW; ++t8) {
            const int t = w + TW * t8;
            if (w < TW && t < TRI) {
                int it, jt;
                tri_tile(t, it, jt);
                const int i = it * 16 + q * 4, j = jt * 16 + l16;
                const uint32_t flip = flip_of<T>((it + jt) & 1);
                frag yf[2], xf[2];
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    yf[ks] = read_rows(sh.y, XLD, it * 16, ks * 32, lane);
                    xf[ks] = read_rows(sh.x, XLD, jt * 16, ks * 32, lane);
                }
                const float dj = s_dt[j];
                const f32x4 ex = (*reinterpret_cast<const f32x4 *>(s_cum + i) - s_cum[j]) +
                                 (*reinterpret_cast<const f32x4 *>(s_low + i) - s_low[j]);
                in_order();
                f32x4 dp = {0, 0, 0, 0}, m, wr;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) dp = mma(flipped(yf[ks], flip), xf[ks], dp);
                if (flip) dp = -dp;
                double col = 0.0;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool in = i + r >= j;
                    const float dec = in ? exp2_fast(ex[r]) : 0.0f;
                    if (i + r == j) diag += dp[r];
                    m[r] = in ? sc[t8][r] * dec : 0.0f;
                    const float s = in ? dp[r] * dec * dj : 0.0f;
                    ds[t8][r] += s;
                    wr[r] = i + r == j ? 0.0f : s * sc[t8][r];      // a token's own pair crosses no decay
                    col += wr[r];
                }
                write_split4<NS>(sh.m + j * MLD + i, Q * MLD, m);
                col += __shfl_xor(col, 16);
                col += __shfl_xor(col, 32);
                if (q == 0) sh.col[at][it][j] = col;
                const double row = row_sum4<double>(wr, lane);
                if ((l16 & 3) == 0) sh.row[at][jt][i + (l16 >> 2)] = row;
            }
        }
        Split<T, NS> hs[2];
        float part = 0.0f;
        if (it0 == 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) part = fmaf(h0[e], u[e], part);
        }
        make_split(reinterpret_cast<const float (&)[8]>(h0[0]), hs[0]);
        make_split(reinterpret_cast<const float (&)[8]>(h0[8]), hs[1]);
        const uint32_t flip_s = flip_of<T>(nt & 1);
        const float sign_s = flip_s ? -1.0f : 1.0f;
        part = wave_sum(part);
        diag = wave_sum(diag);
        if (lane == 0) {
            sh.dot[at][w] = part;
            sh.dd[at][w] = diag;
        }
        // dC and dB through the states at the borders
        if (on) {
            frag yf[2], xf[2], uf[2][NS];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int m = 0; m < NS; ++m) uf[ks][m] = read_rows(sh.u + m * SP * ULD, ULD, nt * 16, ks * 32, lane);
            auto read = [&](int i) __attribute__((always_inline)) {
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    yf[ks] = read_rows(sh.y, XLD, (it0 + i) * 16, ks * 32, lane);
                    xf[ks] = read_rows(sh.x, XLD, (it0 + i) * 16, ks * 32, lane);
                }
            };
            read(0);
#pragma unroll
            for (int i = 0; i < ITW; ++i) {
                const int row = (it0 + i) * 16 + q * 4;
                const f32x4 ei = *reinterpret_cast<const f32x4 *>(s_e + row);
                const f32x4 wi = *reinterpret_cast<const f32x4 *>(s_w + row) * *reinterpret_cast<const f32x4 *>(s_dt + row);
                f32x4 cv;
#pragma unroll
                for (int r = 0; r < 4; ++r) cv[r] = (float)sh.c[(row + r) * BLD + nt * 16 + l16];
                in_order();
                f32x4 ac = {0, 0, 0, 0}, ab = {0, 0, 0, 0};
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int m = 0; m < NS; ++m) {
                        ac = mma(flipped(yf[ks], flip_s), hs[ks].f[m], ac);
                        ab = mma(xf[ks], uf[ks][m], ab);
                    }
                if (i + 1 < ITW) read(i + 1);       // under way while the sums follow
                in_order();
                ac *= ei * sign_s;
                dC[i] += ac;
                dB[i] += ab * wi;
                const float s = row_sum4(ac * cv, lane);
                if ((l16 & 3) == 0) sh.cd[at][nt][row + (l16 >> 2)] = s;
            }
        }
        if (w == 7 && k > 0) finish(k - 1);
        __syncthreads();
        if (k + 1 < blocks) {
            fetch_states(k + 1);
            fetch(k + 1);
        }
        // dx
        {
            const uint32_t flip_x = flip_of<T>(pt & 1);
            const float sign_x = flip_x ? -1.0f : 1.0f;
            f32x4 dx[JW];
            frag uf[2][NS], bf[2][JW];
            auto read = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
                for (int m = 0; m < NS; ++m) uf[ks & 1][m] = read_cols(sh.u + m * SP * ULD, ULD, ks * 32, pt * 16, lane);
#pragma unroll
                for (int j = 0; j < JW; ++j) bf[ks & 1][j] = read_rows(sh.b, BLD, (jt0 + j) * 16, ks * 32, lane);
            };
#pragma unroll
            for (int j = 0; j < JW; ++j) dx[j] = f32x4{0, 0, 0, 0};
            read(0);
            frag yf[Q / 32], mf[JW][NS];
            float xv[JW][4], yv[JW][4];
#pragma unroll
            for (int ks = 0; ks < SP / 32; ++ks) {
                if (ks + 1 < SP / 32) {
                    read(ks + 1);
                } else {
#pragma unroll
                    for (int s = 0; s < Q / 32; ++s) yf[s] = read_cols(sh.y, XLD, s * 32, pt * 16, lane);
#pragma unroll
                    for (int j = 0; j < JW; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int o = ((jt0 + j) * 16 + q * 4 + r) * XLD + pt * 16 + l16;
                            xv[j][r] = (float)sh.x[o];
                            yv[j][r] = (float)sh.y[o];
                        }
                }
                in_order();
#pragma unroll
                for (int m = 0; m < NS; ++m)
#pragma unroll
                    for (int j = 0; j < JW; ++j) dx[j] = mma(flipped(bf[ks & 1][j], flip_x), uf[ks & 1][m], dx[j]);
                in_order();
            }
#pragma unroll
            for (int j = 0; j < JW; ++j) {
                dx[j] *= *reinterpret_cast<const f32x4 *>(s_w + (jt0 + j) * 16 + q * 4);
                // what comes from behind the chunk, for dl: as the whole less the
                // chunk's own part it would lose the digits that ddt_bias sums up
                const f32x4 xi = {xv[j][0] * dx[j][0], xv[j][1] * dx[j][1], xv[j][2] * dx[j][2], xv[j][3] * dx[j][3]};
                const float s = row_sum4(xi, lane);
                if ((l16 & 3) == 0) sh.xi[pt][(jt0 + j) * 16 + q * 4 + (l16 >> 2)] = s * sign_x;
            }
            // M's tiles (i >= j): in the upper half of the tokens only the second 32 meet it
#pragma unroll
            for (int ks = 0; ks < Q / 32; ++ks) {
                if (ks * 2 + 1 < jt0) continue;
#pragma unroll
                for (int j = 0; j < JW; ++j)
#pragma unroll
                    for (int m = 0; m < NS; ++m)
                        mf[j][m] = read_rows(sh.m + m * Q * MLD, MLD, (jt0 + j) * 16, ks * 32, lane);
                in_order();
#pragma unroll
                for (int m = 0; m < NS; ++m)
#pragma unroll
                    for (int j = 0; j < JW; ++j) dx[j] = mma(mf[j][m], flipped(yf[ks], flip_x), dx[j]);
            }
#pragma unroll
            for (int j = 0; j < JW; ++j) {
                const f32x4 dj = *reinterpret_cast<const f32x4 *>(s_dt + (jt0 + j) * 16 + q * 4);
                f32x4 xd;
                dx[j] *= sign_x;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = (jt0 + j) * 16 + q * 4 + r;
                    xd[r] = xv[j][r] * dx[j][r];
                    // in place of x: nothing reads other waves' columns of it any more
                    sh.x[row * XLD + pt * 16 + l16] = (T)fmaf(skip, yv[j][r], dj[r] * dx[j][r]);
                }
                const float s = row_sum4(xd, lane);
                if ((l16 & 3) == 0) sh.xd[pt][(jt0 + j) * 16 + q * 4 + (l16 >> 2)] = s;
            }
        }
        if (w == 6 && k + 1 < blocks && (k + 1) % p.NPB == 0) decays(k + 1);
        __syncthreads();
        const int64_t base = fresh_scalar(base_);
        XT::write(sh.x, (T *)p.dx + base * p.dx_ld + (int64_t)h * p.P + pb * kPB, p.dx_ld, rows, all_rows,
                  pcols, p.vec);
    }
    if (w == 7) finish(blocks - 1);
    // the parts of dB and dC inside the chunk, from the sum of dS over the heads
    // (M's last readers are behind the barrier above)
#pragma unroll
    for (int k = 0; k < TPW; ++k) {
        const int t = w + TW * k;
        if (w < TW && t < TRI) {
            int it, jt;
            tri_tile(t, it, jt);
            write_split4<NS>(sh.m + (jt * 16 + l16) * MLD + it * 16 + q * 4, Q * MLD, ds[k]);
        }
    }
    __syncthreads();
    if (!on) return;
#pragma unroll
    for (int ks = 0; ks < Q / 32; ++ks) {
        const frag bf = read_cols(sh.b, BLD, ks * 32, nt * 16, lane), cf = read_cols(sh.c, BLD, ks * 32, nt * 16, lane);
#pragma unroll
        for (int i = 0; i < ITW; ++i)
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                const T *s = sh.m + m * Q * MLD;
                const int t = it0 + i;
                if (t < 2 * ks + 2) dB[i] = mma(read_rows(s, MLD, t * 16, ks * 32, lane), cf, dB[i]);
                if (t >= 2 * ks) dC[i] = mma(read_cols(s, MLD, ks * 32, t * 16, lane), bf, dC[i]);
            }
    }
    const int s = nt * 16 + l16;
    if (s >= p.S) return;
#pragma unroll
    for (int i = 0; i < ITW; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = (it0 + i) * 16 + q * 4 + r;
            if (row >= all_rows) continue;
            if (row >= rows) dB[i][r] = dC[i][r] = 0.0f;
            if (p.slices == 1) {
                ((T *)p.db)[(base_ + row) * p.db_ld + g * p.S + s] = (T)dB[i][r];
                ((T *)p.dc)[(base_ + row) * p.dc_ld + g * p.S + s] = (T)dC[i][r];
            } else {
                const int64_t o = (((int64_t)slice * p.N * p.L + base_ + row) * p.G + g) * SP + s;
                p.part_b[o] = dB[i][r];
                p.part_c[o] = dC[i][r];
            }
        }
}

// What the chunks and head slices left: the first 3 H workgroups add dA,
// ddt_bias and dD of a head over the chunks, the others dB and dC over the head
// slices, all in a fixed order.
template <typename T, int SP>
__global__ void __launch_bounds__(256) scan_reduce_kernel(ScanParams p, float *da, float *dbias, float *dd)
{
    if (blockIdx.x < 3u * p.H) {
        __shared__ double red[256];
        const int which = blockIdx.x / p.H, h = blockIdx.x - which * p.H;
        const int64_t NK = (int64_t)p.N * p.K;
        float *out = which == 0 ? da : which == 1 ? dbias : dd;
        if (!out) return;
        double s = 0.0;
        for (int64_t i = threadIdx.x; i < NK; i += 256) s += p.part_head[(which * NK + i) * p.H + h];
        red[threadIdx.x] = s;
        __syncthreads();
        for (int o = 128; o > 0; o >>= 1) {
            if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
            __syncthreads();
        }
        if (threadIdx.x == 0) out[h] = (float)red[0];
        return;
    }
    const int64_t id = ((int64_t)blockIdx.x - 3 * p.H) * 256 + threadIdx.x, rows = (int64_t)p.N * p.L * p.G;
    if (id >= rows * SP) return;
    const int64_t rg = id / SP, row = rg / p.G;
    const int s = (int)(id - rg * SP), g = (int)(rg - row * p.G);
    if (s >= p.S) return;
    float b = 0.0f, c = 0.0f;
#pragma unroll 4
    for (int k = 0; k < p.slices; ++k) {
        b += p.part_b[k * rows * SP + id];
        c += p.part_c[k * rows * SP + id];
    }
    ((T *)p.db)[row * p.db_ld + g * p.S + s] = (T)b;
    ((T *)p.dc)[row * p.dc_ld + g * p.S + s] = (T)c;
}

// ---- one token -----------------------------------------------------------------
// The state is read and written once, 8 bytes for 5 flop: HBM bounds it, and at
// one sequence the launch does.  A wave takes kStepRows groups of channels; in a
// group 64 / LPR channels lie beside each other, LPR lanes with V neighbouring
// states each, so a wave's accesses are whole lines and y's sum is a few
// exchanges between lanes.  64 sequences x 64 heads x 64 x 128 (269 MB): 54 us, 5.0
// TB/s, the rate of a large copy (5.1); 57 without the hint on the stores, 67 with
// two rows.  One sequence of 32 heads: 5.7 us.
constexpr int kStepRows = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanParams p, int lpr, int blocks)
{
    constexpr int V = 4;
    const int lane = threadIdx.x & 63, w = wave_id();
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
                if (s0 < p.S) stream_f32<float, V>(s, st[k]);
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
