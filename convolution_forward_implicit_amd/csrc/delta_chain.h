// The passes of the gated delta rule that go from chunk to chunk: the states with y,
// the states for a gradient, and the states' gradient.
//
// A chunk's state follows from the one before it by three products, each of which needs
// all of the one before: K S0^T gives Z, N (beta Z) gives Y, K^T U the new state.  With few
// heads this chain is what takes the time, so a workgroup has 16 channels of one head
// only (two blocks of 16 where there are enough for all compute units, each product for
// both before the barrier) and its four waves share every product: wave t has the tokens
// 16 t .. of the first two and, of the third, the keys 32 t .. (and 128 on), whose state it
// holds.  What each leaves goes to the others through LDS, split into its terms once,
// with a barrier behind each product.  Four more waves do what the chain does not wait
// for: they bring K and N into LDS two chunks ahead and compute y or, going back, what
// M^T dO and Q^T dO add; their own operands (Q and M) have one reader each and go to its
// registers.
//
// A chunk of 128 keys takes 1.85 us: a third of it the three splits and their way through
// LDS, a quarter the matrix instructions (33 of a wave one behind the other), the rest
// barriers and reads of LDS.  K S0^T by the keys whose state a wave holds, summed through
// LDS instead of the state's terms read by all, took 5% less with 128 keys and 10 to 20%
// more with 64 and fewer.
#pragma once

#include "delta_kernels.h"
#include "igemm_dma.h"

namespace convfwd {

enum ChainMode { CHAIN_Y, CHAIN_STATES, CHAIN_BACK };

constexpr int kHelpers = 4;

template <typename T, int SP, ChainMode MODE, int CB> struct ChainShared {
    static constexpr int KS = SP / 32, NT = kN<T>;
    static constexpr int KEYS = 4 * KS * kFrag<T>, TRI = kTri * NT * kFrag<T>, OPS = KEYS + kRows + TRI;
    struct Exchange {
        char s[NT * KS * kFrag<T>];     // the state (its gradient)
        char a[NT * 2 * kFrag<T>];      // Z (dU)
        char b[NT * 2 * kFrag<T>];      // e^{c_Q - c} U (e^c dV)
        char y[2][(MODE == CHAIN_Y ? NT : 0) * 2 * kFrag<T> + 16];      // Y of this chunk and the last
        f32x4 in[2][4][64];             // V (M^T dO) of this chunk and the next
        f32x4 ds[MODE == CHAIN_BACK ? SP / 16 : 0][64];                 // scale (e^c dO)^T Q
    };
    static constexpr int LEFT = 160 * 1024 - CB * (int)sizeof(Exchange);
    // chunks of K and N: the one in use and those under way
    static constexpr int NB = LEFT / OPS >= 3 ? 3 : LEFT / OPS;
    static constexpr int LEAST = KEYS / 1024 / kHelpers + TRI / 1024 / kHelpers;     // loads of a chunk that every helper starts
    __align__(16) char ops[NB][OPS];
    __align__(16) Exchange x[CB];
};

// KB kilobytes of memory to LDS, by the helpers.  The loads are written out: the
// compiler, which cannot see what they write, would wait for them before any read of
// LDS.  K and Q come as the preparation laid them out: from their rows, 64 bytes of
// each at a time, y took 18 us of 110 more (32 heads, 4096 tokens) and the preparation
// 1 of 32 less.
template <int KB> SEQ_DEV void fetch(const char *from, char *to, int wave, int lane)
{
    const i32x4_t buf = uniform_rsrc(buffer_rsrc(from, KB * 1024));
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)to);
#pragma unroll
    for (int e = 0; e < KB; e += kHelpers) {
        const uint32_t b = (uint32_t)(e + wave) * 1024;
        uint32_t saved;
        if (KB % kHelpers == 0 || e + wave < KB)
            asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
                         : "=&s"(saved) : "s"(at + b), "v"(lane * 16), "s"(buf), "s"(b) : "memory");
    }
}
// The workgroup's waves meet; LDS writes are done, loads may be under way.
SEQ_DEV void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The four rows 4q + r of a column that a lane of a result holds, of `rows` rows of a
// tensor from row `first`: rows behind and columns at P and behind come as zeros and are
// not written.
template <typename T> struct LaneRows {
    __amdgpu_buffer_rsrc_t buf;
    uint32_t at, step;
    SEQ_DEV LaneRows(const void *g, int64_t ld, int64_t first, int rows, int P, int ch, int lane)
    {
        const int64_t bytes = rows > 0 ? ((int64_t)(rows - 1) * ld + P) * (int64_t)sizeof(T) : 0;
        buf = __builtin_amdgcn_make_buffer_rsrc((T *)const_cast<void *>(g) + first * ld, 0, (int)bytes, 0x00020000);
        step = (uint32_t)ld * (uint32_t)sizeof(T);
        at = ch < P ? (uint32_t)((lane >> 4) * 4) * step + (uint32_t)ch * (uint32_t)sizeof(T) : 0x80000000u;
    }
    SEQ_DEV uint32_t bits(int r) const      // an element's, as a float's
    {
        if constexpr (sizeof(T) == 4) return __builtin_amdgcn_raw_buffer_load_b32(buf, at + (uint32_t)r * step, 0, 0);
        else return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(buf, at + (uint32_t)r * step, 0, 0) << 16;
    }
    SEQ_DEV void put(int r, float v) const
    {
        if constexpr (sizeof(T) == 4)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), buf, at + (uint32_t)r * step, 0, kStream);
        else
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)v), buf, at + (uint32_t)r * step, 0, kStream);
    }
};

// A result of the tokens 16 t .. as terms of an operand over the tokens: half of the 32
template <typename T, int NS> SEQ_DEV void put_half(char *at, int t, int lane, f32x4 v)
{
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<f32x4 *>(at + (t >> 1) * kFrag<T> + (t & 1) * 1024)[lane] = v;
    } else {
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            float a = v[0], b = v[1], c = v[2], d = v[3];
            const uint32_t lo = take_pair(a, b), hi = take_pair(c, d);
            v = f32x4{a, b, c, d};
            *reinterpret_cast<uint64_t *>(at + (k * 2 + (t >> 1)) * kFrag<T> + lane * 16 + (t & 1) * 8) = (uint64_t)hi << 32 | lo;
        }
    }
}
template <typename T, int NS> SEQ_DEV void get_split(const char *at, int apart, int lane, Split<T, NS> &s)
{
#pragma unroll
    for (int e = 0; e < NS; ++e) s.f[e] = get_frag<T>(at + e * apart, lane);
}
// K^T's operand of the keys 32 s + 8 (r / 4) + 4 a + r % 4 (row r) and the tokens 32 P + 4q ..,
// 32 P + 16 + 4q .. from K's in LDS, [4][KS]
template <int KS> SEQ_DEV bf16x8 get_transposed(const char *at, int P, int s, int a, int lane, bf16_t)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
    const int i = lane & 15;
    const char *p = at + (2 * P * KS + s) * 1024 + ((i & 3) * 16 + (lane >> 4) * 4 + (i >> 2)) * 16 + 8 * a;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + KS * 1024));
    return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int KS> SEQ_DEV Frag<float>::type get_transposed(const char *at, int P, int s, int a, int lane, float)
{
    const int r = lane & 15;
    // key 8 (r / 4) + 4 a + r % 4 of token row: lane group r / 4, vector a, element r % 4
    const float *p = reinterpret_cast<const float *>(at + (2 * P * KS + s) * 2048 + a * 1024 + ((r >> 2) * 16 + (lane >> 4) * 4) * 16) + (r & 3);
    Frag<float>::type f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = p[e * 4], f.v[4 + e] = p[KS * 512 + e * 4];
    return f;
}

template <typename T, int SP, ChainMode MODE, int CB>
SEQ_DEV void delta_chain(const DeltaParams &p, int64_t unit, ChainShared<T, SP, MODE, CB> &sh)
{
    typedef ChainShared<T, SP, MODE, CB> Shared;
    constexpr bool GRAD = MODE != CHAIN_Y, BACK = MODE == CHAIN_BACK;
    constexpr int KS = SP / 32, NT = kN<T>, NB = Shared::NB, KEYS = Shared::KEYS, F = kFrag<T>;
    constexpr int OWN = (KS + 3) / 4;                   // key blocks that a wave may hold
    const int lane = threadIdx.x & 63, w = wave_id(), l16 = lane & 15, q4 = (lane >> 4) * 4;
    const int64_t nh = unit / p.blocks, n = nh / p.H;
    const int h = (int)(nh - n * p.H), grp = h / (p.H / p.G), ch0 = (int)(unit - nh * p.blocks) * 16 * CB + l16;
    const int64_t len = seq_len(p.lengths, n, p.L);
    const int live = (int)((len + kDQ - 1) / kDQ);
    const char *keys = p.keys + (n * p.K * p.G + grp) * keys_bytes<T, SP>(GRAD), *heads = p.heads + (n * p.K * p.H + h) * head_bytes<T>(GRAD);
    const int64_t keys_step = p.G * keys_bytes<T, SP>(GRAD), head_step = p.H * head_bytes<T>(GRAD);
    constexpr int64_t tri = (GRAD ? (int64_t)sizeof(ChunkScalars) : kRows) + (BACK ? Shared::TRI : 0);      // N, or its transpose
    auto chunk = [&](int i) { return BACK ? live - 1 - i : i; };
    const int t = w & 3;
    // rows 16 t .. of this chunk
    auto rows_of = [&](const void *x, int64_t ld, int i, int tile, int c) {
        const int64_t t0 = (int64_t)chunk(i) * kDQ + 16 * tile;
        return LaneRows<T>((const T *)x + (int64_t)h * p.P, ld, n * p.L + t0, (int)(len - t0 < 16 ? len - t0 : 16), p.P, ch0 + 16 * c, lane);
    };
    if (w >= 4) {
        auto load = [&](int i) {
            const char *k = keys + chunk(i) * keys_step, *a = heads + chunk(i) * head_step;
            fetch<KEYS / 1024>(k, sh.ops[i % NB], t, lane);
            fetch<kRows / 1024>(a, sh.ops[i % NB] + KEYS, t, lane);
            fetch<Shared::TRI / 1024>(a + tri, sh.ops[i % NB] + KEYS + kRows, t, lane);
        };
        constexpr int NQ = BACK ? 4 * OWN : MODE == CHAIN_Y ? KS : 0, TM = MODE == CHAIN_STATES ? 0 : NT;
        typename Frag<T>::type qf[NQ + 1];
        Split<T, TM + 1> mf[2];
        uint32_t vb[CB][16];            // the next dO, or v
        auto load_q = [&](int i) {
            const char *k = keys + chunk(i) * keys_step;
#pragma unroll
            for (int s = 0; s < NQ; ++s) {
                if (!BACK) qf[s] = get_frag<T>(k + ((4 + t) * KS + s) * F, lane);
                else if (t + 4 * (s >> 2) < KS) qf[s] = get_frag<T>(k + (12 * KS + (t + 4 * (s >> 2)) * 4 + (s & 3)) * F, lane);
            }
        };
        auto load_m = [&](int i) {
            const char *m = heads + chunk(i) * head_step + tri + Shared::TRI;
#pragma unroll
            for (int P = 0; P < 2; ++P)
                if (BACK ? P >= t / 2 : P <= t / 2) {
#pragma unroll
                    for (int e = 0; e < TM; ++e)
                        mf[P].f[e] = get_frag<T>(m + ((BACK ? upper(t, P) : lower(t, P)) * NT + e) * F, lane);
                }
        };
        auto load_v = [&](int i) {
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                const LaneRows<T> rows = rows_of(p.v, p.v_ld, i, t, c);
#pragma unroll
                for (int r = 0; r < 4; ++r) vb[c][r] = rows.bits(r);
            }
        };
        auto put_v = [&](int i) {
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                f32x4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t b = vb[c][r];
                    v[r] = __builtin_bit_cast(float, b);
                }
                sh.x[c].in[i & 1][t][lane] = v;
            }
        };
        f32x4 dy[CB][4];
        auto load_dy = [&](int i) {
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const LaneRows<T> rows = rows_of(p.dy, p.dy_ld, i, e, c);
#pragma unroll
                    for (int r = 0; r < 4; ++r) vb[c][4 * e + r] = rows.bits(r);
                }
        };
        auto take_dy = [&]() {
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t b = vb[c][e];
                    dy[c][e / 4][e % 4] = __builtin_bit_cast(float, b);
                }
        };
        auto put_du = [&](int i) {      // M^T dO of chunk i, whose dO is in dy
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                Split<T, 1> d[2];
                stack(dy[c][0], dy[c][1], d[0]);
                stack(dy[c][2], dy[c][3], d[1]);
                f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
                for (int P = 0; P < 2; ++P)
                    if (P >= t / 2) {
#pragma unroll
                        for (int e = TM - 1; e >= 0; --e) acc[P] = mma(mf[P].f[e], d[P].f[0], acc[P]);
                    }
                sh.x[c].in[i & 1][t][lane] = acc[0] + acc[1];
            }
        };
        // y's part by the chunk's own tokens, and its rows
        auto put_y = [&](int i, const f32x4 (&y)[CB]) {
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                f32x4 acc[2] = {y[c], f32x4{0, 0, 0, 0}};
#pragma unroll
                for (int P = 0; P < 2; ++P)
                    if (P <= t / 2) {
                        Split<T, NT> b;
                        get_split(sh.x[c].y[i & 1] + P * F, 2 * F, lane, b);
#pragma unroll
                        for (int e = 0; e < NT; ++e)
#pragma unroll
                            for (int k = 0; k < NT - e; ++k) acc[P] = mma(mf[P].f[e], b.f[k], acc[P]);
                    }
                const LaneRows<T> rows = rows_of(p.y, p.y_ld, i, t, c);
                const f32x4 sum = acc[0] + acc[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) rows.put(e, sum[e]);
            }
        };
        if (NB > 1 && live > 0) load(0);
        if (NB > 2 && live > 1) load(1);
        if (live > 0) {
            load_q(0);
            if constexpr (BACK) {
                load_m(0);
                load_dy(0);
                take_dy();
                put_du(0);
                if (live > 1) load_dy(1), load_m(1);
            } else {
                load_v(0);
                put_v(0);
                if (live > 1) load_v(1);
            }
        }
        f32x4 y[CB], last[CB];
        for (int i = 0; i < live; ++i) {
            const ChunkScalars *cs = reinterpret_cast<const ChunkScalars *>(sh.ops[i % NB] + KEYS);
            if (NB == 1) {
                meet();
                load(i);
            }
            // This chunk's K and N are there.  Behind their loads came those of the next one's and, at least, Q, v and
            // a block of M (going back a block of M^T and dO), which may be under way.
            if (NB < 3 || i == 0 || i + 1 >= live) wait_vmcnt<0>();
            else wait_vmcnt<(MODE == CHAIN_Y ? NQ + TM + 4 * CB : BACK ? TM + 16 * CB : 4 * CB) + Shared::LEAST>();
            meet();
            if (NB == 2 && i + 1 < live) load(i + 1);
            // A chunk's y is finished while the next one is under way: beside its second product, the shortest of the
            // three; beside the third, which all of the chain waits for, the pass took 131 us instead of 119.
            if constexpr (MODE == CHAIN_Y) {
                const f32x4 grow = *reinterpret_cast<const f32x4 *>(cs->from_start + 16 * t + q4);
#pragma unroll
                for (int c = 0; c < CB; ++c) {
                    last[c] = y[c];
                    f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        Split<T, NT> b;
                        get_split(sh.x[c].s + s * F, KS * F, lane, b);
#pragma unroll
                        for (int e = 0; e < NT; ++e) acc[s & 1] = mma(qf[s], b.f[e], acc[s & 1]);
                    }
                    y[c] = (acc[0] + acc[1]) * (grow * p.scale);
                }
                if (i + 1 < live) load_q(i + 1);
                meet();
                if (i + 1 < live) put_v(i + 1);
                load_v(i + 2 < live ? i + 2 : i);
                if (i > 0) put_y(i - 1, last);
                load_m(i);
                meet();
                if (NB == 3 && i + 2 < live) load(i + 2);
            }
            if constexpr (BACK) {
                // (scale e^c dO)^T Q for the states of wave t
#pragma unroll
                for (int c = 0; c < CB; ++c) {
                    Split<T, NT> x[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dy[c][e] = dy[c][e] * (*reinterpret_cast<const f32x4 *>(cs->from_start + 16 * e + q4) * p.scale);
                    stack(dy[c][0], dy[c][1], x[0]);
                    stack(dy[c][2], dy[c][3], x[1]);
#pragma unroll
                    for (int o = 0; o < OWN; ++o) {
                        if (t + 4 * o >= KS) continue;
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
                            for (int e = NT - 1; e >= 0; --e)
#pragma unroll
                                for (int P = 0; P < 2; ++P) acc[P] = mma(qf[4 * o + 2 * a + P], x[P].f[e], acc[P]);
                            sh.x[c].ds[2 * (t + 4 * o) + a][lane] = acc[0] + acc[1];
                        }
                    }
                }
                if (i + 1 < live) load_q(i + 1);
                meet();
                if (i + 1 < live) {
                    take_dy();
                    put_du(i + 1);
                }
                if (i + 2 < live) load_m(i + 2), load_dy(i + 2);
                meet();
                if (NB == 3 && i + 2 < live) load(i + 2);
            }
            if constexpr (MODE == CHAIN_STATES) {
                meet();
                if (i + 1 < live) put_v(i + 1);
                load_v(i + 2 < live ? i + 2 : i);
                meet();
                if (NB == 3 && i + 2 < live) load(i + 2);
            }
        }
        if (MODE == CHAIN_Y && live > 0) put_y(live - 1, y);
        for (int ch = ch0; MODE == CHAIN_Y && ch < p.P && ch < ch0 + 16 * CB; ch += 16)
            for (int64_t r = len + 4 * t + (lane >> 4); r < p.L; r += 16) ((T *)p.y)[(n * p.L + r) * p.y_ld + (int64_t)h * p.P + ch] = (T)0.0f;
        return;
    }
    f32x4 st[CB][OWN][2];
    auto state_at = [&](int o, int a, int r) { return 32 * (t + 4 * o) + 2 * q4 + 4 * a + r; };      // the key
    const float *from = BACK ? p.dstate_out : p.state;
#pragma unroll
    for (int c = 0; c < CB; ++c) {
        const float *g = from + (nh * p.P + ch0 + 16 * c) * p.S;
#pragma unroll
        for (int o = 0; o < OWN; ++o)
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    st[c][o][a][r] = from && ch0 + 16 * c < p.P && state_at(o, a, r) < p.S ? g[state_at(o, a, r)] : 0.0f;
    }
    auto put_state = [&](int c) {
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            if (t + 4 * o >= KS) continue;
            Split<T, NT> s;
            stack(st[c][o][0], st[c][o][1], s);
#pragma unroll
            for (int e = 0; e < NT; ++e) put_frag(sh.x[c].s + (e * KS + t + 4 * o) * F, lane, s.f[e]);
        }
    };
    if (live > 0)
#pragma unroll
        for (int c = 0; c < CB; ++c) put_state(c);
    for (int i = 0; i < live; ++i) {
        const char *ops = sh.ops[i % NB], *tr = ops + KEYS + kRows;
        const ChunkScalars *cs = reinterpret_cast<const ChunkScalars *>(ops + KEYS);
        const int64_t at = nh * p.K + chunk(i);
        if (NB == 1) meet();
        meet();
        const f32x4 grow = *reinterpret_cast<const f32x4 *>(cs->from_start + 16 * t + q4);
        const f32x4 fade = *reinterpret_cast<const f32x4 *>(cs->to_end + 16 * t + q4);
        const f32x4 beta = *reinterpret_cast<const f32x4 *>(cs->beta + 16 * t + q4);
        const float total = cs->from_start[kDQ - 1];
        typename Frag<T>::type kf[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) kf[s] = get_frag<T>(ops + (t * KS + s) * F, lane);
        Split<T, NT> nf[2];
        typename Frag<T>::type kt[OWN][2][2];
        f32x4 z[CB];
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            // K S0^T, a sum of each term by itself
            Split<T, NT> sp[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) get_split(sh.x[c].s + s * F, KS * F, lane, sp[s]);
            const f32x4 in = sh.x[c].in[i & 1][t][lane];
            if (c == 0) {
                // what the next products read of K and N, so that no wait for it stands in front of a barrier
#pragma unroll
                for (int P = 0; P < 2; ++P)
                    if (BACK ? P >= t / 2 : P <= t / 2) get_split(tr + (BACK ? upper(t, P) : lower(t, P)) * NT * F, F, lane, nf[P]);
#pragma unroll
                for (int o = 0; o < OWN; ++o)
                    if (t + 4 * o < KS)
#pragma unroll
                        for (int a = 0; a < 2; ++a)
#pragma unroll
                            for (int P = 0; P < 2; ++P) kt[o][a][P] = get_transposed<KS>(ops, P, t + 4 * o, a, lane, T());
            }
            f32x4 r[NT];
#pragma unroll
            for (int e = 0; e < NT; ++e) r[e] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int e = 0; e < NT; ++e) r[e] = mma(kf[s], sp[s].f[e], r[e]);
#pragma unroll
            for (int e = NT - 1; e > 0; --e) r[e - 1] = r[e - 1] + r[e];
            z[c] = BACK ? in + r[0] * fade : in - grow * r[0];          // dU, Z
            put_half<T, NT>(sh.x[c].a, t, lane, z[c]);
            if constexpr (GRAD) {
                float *b = p.bound[BACK] + at * states_floats(p.PP, SP) + (int64_t)(ch0 + 16 * c) * SP + 2 * q4;
#pragma unroll
                for (int o = 0; o < OWN; ++o)
                    if (t + 4 * o < KS)
#pragma unroll
                        for (int a = 0; a < 2; ++a) *reinterpret_cast<f32x4 *>(b + 32 * (t + 4 * o) + 4 * a) = st[c][o][a];
            }
        }
        meet();
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            // N (beta Z); sums that do not wait for each other
            f32x4 acc[2][2] = {{z[c], f32x4{0, 0, 0, 0}}, {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}}};
#pragma unroll
            for (int P = 0; P < 2; ++P)
                if (BACK ? P >= t / 2 : P <= t / 2) {
                    Split<T, NT> b;
                    get_split(sh.x[c].a + P * F, 2 * F, lane, b);
#pragma unroll
                    for (int e = NT - 1; e >= 0; --e)
#pragma unroll
                        for (int k = 0; k < NT - e; ++k) acc[P][e + k < NT - 1] = mma(nf[P].f[e], b.f[k], acc[P][e + k < NT - 1]);
                }
            z[c] = (acc[0][0] + acc[1][0]) + (acc[0][1] + acc[1][1]);
            put_half<T, NT>(sh.x[c].b, t, lane, z[c] * (BACK ? beta * grow * -1.0f : beta * fade));
            if constexpr (MODE == CHAIN_Y) put_half<T, NT>(sh.x[c].y[i & 1], t, lane, z[c]);
        }
        meet();
        // the state behind the chunk
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            if (t >= KS) break;
            Split<T, NT> u[2];
#pragma unroll
            for (int P = 0; P < 2; ++P) get_split(sh.x[c].b + P * F, 2 * F, lane, u[P]);
            f32x4 sums[OWN][2][2];
#pragma unroll
            for (int o = 0; o < OWN; ++o)
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    sums[o][a][0] = st[c][o][a] * total;
                    sums[o][a][1] = f32x4{0, 0, 0, 0};
                    if constexpr (BACK) {
                        if (t + 4 * o < KS) sums[o][a][1] = sh.x[c].ds[2 * (t + 4 * o) + a][lane];
                    }
                }
#pragma unroll
            for (int e = NT - 1; e >= 0; --e)
#pragma unroll
                for (int P = 0; P < 2; ++P)
#pragma unroll
                    for (int o = 0; o < OWN; ++o) {
                        if (t + 4 * o >= KS) continue;
#pragma unroll
                        for (int a = 0; a < 2; ++a) sums[o][a][1 - P] = mma(kt[o][a][P], u[P].f[e], sums[o][a][1 - P]);
                    }
#pragma unroll
            for (int o = 0; o < OWN; ++o)
#pragma unroll
                for (int a = 0; a < 2; ++a) st[c][o][a] = sums[o][a][0] + sums[o][a][1];
            put_state(c);
        }
        if constexpr (GRAD) {
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) p.rows[BACK][at * rows_floats(p.PP) + (16 * t + q4 + e) * p.PP + ch0 + 16 * c] = z[c][e];
        }
    }
    float *to = BACK ? p.dstate : p.state_out;
#pragma unroll
    for (int c = 0; c < CB; ++c)
        if (to && ch0 + 16 * c < p.P)
#pragma unroll
            for (int o = 0; o < OWN; ++o)
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (t + 4 * o < KS && state_at(o, a, e) < p.S)
                            to[(nh * p.P + ch0 + 16 * c) * p.S + state_at(o, a, e)] = st[c][o][a][e];
}

constexpr int kChainThreads = 64 * (4 + kHelpers);

// Keys up to which a workgroup may have two blocks of 16 channels: the exchange of both
// leaves room for a chunk of K and N.
constexpr int kMostPaired = 128;

template <typename T, int SP, int CB> __global__ void __launch_bounds__(kChainThreads) delta_y_kernel(DeltaParams p)
{
    __shared__ ChainShared<T, SP, CHAIN_Y, CB> sh;
    const int64_t units = (int64_t)p.N * p.H * p.blocks, unit = unit_of(blockIdx.x, units);
    if (unit < units) delta_chain<T, SP, CHAIN_Y, CB>(p, unit, sh);
}

// The two passes over the states of a gradient, which do not depend on each other.
template <typename T, int SP, int CB> __global__ void __launch_bounds__(kChainThreads) delta_states_kernel(DeltaParams p)
{
    __shared__ union Both {
        ChainShared<T, SP, CHAIN_STATES, CB> ahead;
        ChainShared<T, SP, CHAIN_BACK, CB> back;
        SEQ_DEV Both() {}
    } sh;
    const int64_t units = (int64_t)p.N * p.H * p.blocks, half = gridDim.x / 2;
    const bool back = blockIdx.x < half;
    const int64_t unit = unit_of(back ? blockIdx.x : blockIdx.x - half, units);
    if (unit >= units) return;
    if (back) delta_chain<T, SP, CHAIN_BACK, CB>(p, unit, sh.back);
    else delta_chain<T, SP, CHAIN_STATES, CB>(p, unit, sh.ahead);
}

}  // namespace convfwd
