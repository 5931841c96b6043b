// Operands and results of the matrix instructions as the sequence kernels hold
// them (16x16 blocks, 64 lanes, q = lane / 16): an operand's lane holds 8 values
// of the reduction for row (or column) lane % 16, a result's lane four rows
// 4q..4q+3 of column lane % 16.  fp32 values enter bf16 products as the sum of
// up to three bf16 numbers.  Also tiles of tensors on their way through LDS, and
// sums over the lanes of a wave.
#pragma once

#include "seq_common.h"

namespace convfwd {

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

}  // namespace convfwd
