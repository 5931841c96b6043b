// The scan's state and forward kernels for bf16 tensors of whole 16-byte rows:
// the formulas and the fragments of scan_kernels.h, fed by direct-to-LDS loads.
//
// scan_kernels.h's forward takes a chunk through one workgroup of four waves:
// tiles through registers into LDS, scores, a barrier, the products with M.  Here
// a ring of three stages is filled by loads that need no registers, two chunks
// ahead, and the waves have jobs that do not wait for each other within a chunk:
//
//   waves 0-3 ("state", 16 channels each):  y' = e^{c_i} h_0 C_i, then the state's update
//   waves 4-7 ("score", 16 tokens each):    M from C . B, y'' = (M + D) x
//
// (wave 4, with the least of the scores, also starts the loads, waves 5 and 6 do
// the decays; eight waves leave each 256 registers to read fragments ahead)
// The score waves' products need no LDS for M: the scores' result blocks are
// the operand of M x as they stand.  y' crosses through LDS, the score waves
// add y'' and store the rows while the next chunk is under way, so there is one
// barrier a chunk.
//
// A load writes 1 KB to LDS in lane order, so rows cannot be padded one by one;
// but each load's 1 KB may lie anywhere and hold any rows: load g of a tile takes
// the rows g, g + G, g + 2G .. (G loads to a tile) and its kilobyte starts 32
// bytes (8 banks) behind the last one's end.  An address is then a lane's
// constant plus a constant, and reads run at the rate of the banks: measured per
// wave instruction, 16 rows of 16 bytes 4.0 clocks (8.0 with 16 or 48 bytes
// between; 8 bytes of each row instead: 16), the transposing read 2.5 (4.0).
//
// What bounds it: 16384 tokens x 64 heads of 64 x 128 (34 Gflop by the recurrence,
// 133 as the products that the splits make of it) take 196-218 us, 3.1 us a chunk
// and workgroup: the matrix unit is busy for a third of that and other vector
// instructions for half, and the two hardly overlap -- a wave of products and a wave
// of FMAs on one SIMD take as long as one after the other (8 products and 24 FMAs:
// 227 clocks, 128 and 107 alone).  LDS is busy for a quarter.  The pass over the
// states is another 62-70 us; back to back the two take 226 us, the registers' forms
// 300.  With two terms for M and h and one number for c_i they took 205 and had lost
// digits: see scan_kernels.h.
#pragma once

#include "igemm_dma.h"
#include "scan_kernels.h"

namespace convfwd {

constexpr int kStages = 3;

// Tiles of 64 tokens x COLS bf16 in that layout
template <int COLS> struct Ring {
    static constexpr int CH = COLS / 8;                  // 16-byte pieces of a row
    static constexpr int LOADS = 64 * COLS * 2 / 1024;   // wave instructions of a tile
    static constexpr int GROUP = (1024 + 32) / 2;        // elements from one load's kilobyte to the next
    static constexpr int BYTES = LOADS * GROUP * 2;

    static SEQ_DEV constexpr int row(int r) { return r % LOADS * GROUP + r / LOADS * COLS; }
    // byte offset into the matrix of what lane `lane` of load `g` fetches
    static SEQ_DEV uint32_t source(int g, int lane, int ld, int cols)
    {
        const int r = g + lane / CH * LOADS, c = (lane & (CH - 1)) * 8;
        return c < cols ? (uint32_t)(r * ld + c) * 2 : kOutOfRange;
    }
    // Row row0 + lane % 16 (row0 a multiple of 16), reduction k0 + 8q ..
    static SEQ_DEV bf16x8 rows(const bf16_t *t, int row0, int k0, int lane)
    {
        return *reinterpret_cast<const bf16x8 *>(t + row(lane & 15) + row(row0) + k0 + (lane >> 4) * 8);
    }
    // Transposing reads over the rows k0 + 4q .. and k0 + 16 + 4q .. (the order of
    // two stacked results; k0 a multiple of 32): lane % 16 = m gets column col0 + m
    // or, spread, the column that makes two results (HALF 0 and 1) an operand whose
    // lane holds 8q .. 8q + 7: col0 + 8 (m / 4) + 4 HALF + m % 4.
    template <bool SPREAD = false, int HALF = 0> static SEQ_DEV bf16x8 cols(const bf16_t *t, int k0, int col0, int lane)
    {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
        const int i = lane & 15, r = (lane >> 4) * 4 + (i >> 2);
        const bf16_t *p = t + row(r) + row(k0) + col0 + (SPREAD ? (i & 3) * 8 + HALF * 4 : (i & 3) * 4);
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + row(16)));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// the state index of row 4q + r of result t of a spread pair
SEQ_DEV int spread_state(int t, int q, int r) { return (t >> 1) * 32 + q * 8 + (t & 1) * 4 + r; }

// the next of the ring's stages
SEQ_DEV int next_stage(int stage, int bytes) { return stage == (kStages - 1) * bytes ? 0 : stage + bytes; }

SEQ_DEV uint32_t lds_address(const void *p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// a chunk's rows of a matrix as a buffer that ends with the last valid element
SEQ_DEV i32x4_t chunk_buffer(const bf16_t *g, int64_t ld, int rows, int cols)
{
    return buffer_rsrc(g, rows > 0 ? (uint32_t)(((rows - 1) * ld + cols) * 2) : 0u);
}

// ---- states ----------------------------------------------------------------------
template <int SP> struct StateDmaShared {
    static constexpr int STAGE = Ring<kPB>::BYTES + Ring<SP>::BYTES;
    __align__(1024) unsigned char ring[kStages * STAGE];
    __align__(16) float w[8][64];       // the weights of eight chunks, four of them in use
    float tot[8];
};

// scan_states of scan_kernels.h
template <int SP, bool REV, bool STORE>
SEQ_DEV void scan_states_dma(const ScanParams &p, int64_t block, StateDmaShared<SP> &sh)
{
    constexpr int Q = 64, NT = SP / 16, STAGE = StateDmaShared<SP>::STAGE;
    typedef Ring<kPB> XR;
    typedef Ring<SP> BR;
    constexpr int ND = (XR::LOADS + BR::LOADS) / 4;         // loads of a wave and chunk
    static_assert(XR::LOADS % 4 == 0 && BR::LOADS % 4 == 0, "whole loads per wave");
    float *seg_state = p.seg_state[REV], *seg_log = p.seg_log[REV];
    const int lane = threadIdx.x & 63, w = wave_id(), q = lane >> 4, l16 = lane & 15;
    const int nseg = STORE ? p.nseg : p.nseg - p.sub;
    const int64_t unit = block / nseg;
    const int s0 = (int)(block - unit * nseg);
    const int seg = STORE ? s0 : REV ? s0 + p.sub : s0;
    const int pb = (int)(unit % p.NPB);
    const int64_t nh = unit / p.NPB, n = nh / p.H;
    const int h = (int)(nh - n * p.H), g = h / (p.H / p.G);
    const int64_t len = seq_len(p.lengths, n, p.L);
    const int pcols = min(kPB, p.P - pb * kPB);
    const int64_t x_ld = REV ? p.dy_ld : p.x_ld, b_ld = REV ? p.c_ld : p.b_ld;
    const bf16_t *xg = (const bf16_t *)(REV ? p.dy : p.x) + n * p.L * x_ld + (int64_t)h * p.P + pb * kPB;
    const bf16_t *bg = (const bf16_t *)(REV ? p.c : p.b) + n * p.L * b_ld + (int64_t)g * p.S;
    const bf16_t *dg = (const bf16_t *)p.dt + n * p.L * p.dt_ld + h;
    const float a = p.a[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
    const int c_lo = seg * p.seg, c_hi = min(p.K, c_lo + p.seg);
    const int c_live = (int)min((int64_t)c_hi, (len + Q - 1) / Q);   // chunks behind the sequence change nothing
    const int steps = max(0, c_live - c_lo);
    const bool busy = w * 16 < pcols;
    const int ch = w * 16 + q * 4;

    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    uint32_t src[ND];
#pragma unroll
    for (int k = 0; k < ND; ++k)
        src[k] = k * 4 < XR::LOADS ? XR::source(k * 4 + w, lane, (int)x_ld, pcols)
                                   : BR::source(k * 4 + w - XR::LOADS, lane, (int)b_ld, p.S);
    auto chunk_of = [&](int k) __attribute__((always_inline)) { return REV ? c_live - 1 - k : c_lo + k; };
    const uint32_t ring = lds_address(sh.ring);
    int fill = 0, stage = 0;        // the stages that the next chunk goes to and is taken from
    auto issue = [&](int k) __attribute__((always_inline)) {
        const int64_t t0 = (int64_t)chunk_of(k) * Q;
        const int rows = (int)min((int64_t)Q, len - t0);
        const i32x4_t xb = chunk_buffer(xg + t0 * x_ld, x_ld, rows, pcols);
        const i32x4_t bb = chunk_buffer(bg + t0 * b_ld, b_ld, rows, p.S);
        const uint32_t to = ring + fill + (uint32_t)w * (2 * XR::GROUP);
#pragma unroll
        for (int i = 0; i < ND; ++i) dma16(i * 4 < XR::LOADS ? xb : bb, src[i], 0, to + i * (8 * XR::GROUP));
        fill = next_stage(fill, STAGE);
    };
    float raw = 0.0f;
    auto fetch_dt = [&](int k) __attribute__((always_inline)) {
        const int64_t t = (int64_t)chunk_of(k) * Q + lane;
        raw = k < steps && t < len ? (float)dg[t * p.dt_ld] + bias : 0.0f;
    };
    // the decays of chunk k, into its slot of eight
    auto decays = [&](int k) __attribute__((always_inline)) {
        float dt;
        double cum;
        chunk_decay(raw, k < steps && (int64_t)chunk_of(k) * Q + lane < len, a, p.softplus, dt, cum);
        const double tot = wave_last(cum);
        sh.w[k & 7][lane] = REV ? exp2_fast((float)cum) : exp2_fast((float)(tot - cum)) * dt;
        if (lane == 0) sh.tot[k & 7] = (float)tot;
    };
    if (steps > 0) {
        fetch_dt(w);
        issue(0);
        if (steps > 1) issue(1);
    }
    if (STORE) start_states<SP, REV>(p, unit, seg, ch, pcols, lane, acc);
    // odd waves carry their states negated: see flipped()
    const uint32_t flip = flip_of<bf16_t>(w & 1);
    const float sign = flip ? -1.0f : 1.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] *= sign;
    float log_dec = 0.0f;
    if (steps > 0) {
        decays(w);
        fetch_dt(4 + w);
        wait_vmcnt<0>();
        __syncthreads();
    }
    for (int k = 0; k < steps; ++k) {
        if (k + 2 < steps) issue(k + 2);        // over chunk k - 1, which all waves are done with
        const bf16_t *sX = (const bf16_t *)(sh.ring + stage), *sB = sX + XR::BYTES / 2;
        stage = next_stage(stage, STAGE);
        if (STORE) {
            float *s = p.bound[REV] + (unit * p.K + chunk_of(k)) * (SP * kPB);
#pragma unroll
            for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4 *>(s + (t * 16 + l16) * kPB + ch) = acc[t] * sign;
        }
        const float tot = sh.tot[k & 7], dec = exp2_fast(tot);
        log_dec += tot;
        if (busy) {
            bf16x8 xf[2], bf[2][NT];
            f32x4 wt[2][2];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                xf[ks] = flipped(XR::cols(sX, ks * 32, w * 16, lane), flip);
                wt[ks][0] = *reinterpret_cast<const f32x4 *>(&sh.w[k & 7][ks * 32 + q * 4]);
                wt[ks][1] = *reinterpret_cast<const f32x4 *>(&sh.w[k & 7][ks * 32 + 16 + q * 4]);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int t = 0; t < NT; ++t) bf[ks][t] = BR::cols(sB, ks * 32, t * 16, lane);
            in_order();
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] *= dec;
            Split<bf16_t, 3> xs[2];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = (float)xf[ks][e] * wt[ks][e / 4][e & 3];
                make_split(v, xs[ks]);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
                for (int m = 0; m < 3; ++m)
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[t] = mma(xs[ks].f[m], bf[ks][t], acc[t]);
            }
        }
        if ((k & 3) == 2) {         // the next four chunks' decays, into the other half of the slots
            decays((k & ~3) + 4 + w);
            fetch_dt((k & ~3) + 8 + w);
        }
        if (k + 2 < steps) wait_vmcnt<ND>();        // loads return in order: at most chunk k + 2's are under way
        else wait_vmcnt<0>();
        __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] *= sign;
    if (!STORE) {
        leave_segment<SP>(p, seg_state, seg_log, unit, seg, ch, lane, log_dec, acc);
    } else if (REV && seg == 0 && p.dstate) {
        float *s = p.dstate + (nh * p.P + pb * kPB) * p.S;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (ch + r < pcols && t * 16 + l16 < p.S) s[(int64_t)(ch + r) * p.S + t * 16 + l16] = acc[t][r];
    }
}

template <int SP, bool STORE> __global__ void __launch_bounds__(256, 2) scan_state_dma_kernel(ScanParams p)
{
    __shared__ StateDmaShared<SP> sh;
    if (blockIdx.x < p.ahead) scan_states_dma<SP, false, STORE>(p, blockIdx.x, sh);
    else scan_states_dma<SP, true, STORE>(p, blockIdx.x - p.ahead, sh);
}

// ---- forward -----------------------------------------------------------------------
template <int SP> struct FwdDmaShared {
    static constexpr int STAGE = Ring<kPB>::BYTES + 2 * Ring<SP>::BYTES;
    __align__(1024) unsigned char ring[kStages * STAGE];       // C, B, x of a chunk
    __align__(16) float y[2][64 * kPB];         // y' of a chunk: token i, piece c of four channels at c ^ i % 16
    __align__(16) float cum[3][64], low[3][64], dt[3][64], w[3][64];    // of three chunks: c_i, its low part, dt_i,
                                                                        // e^{c_Q - c_i} dt_i
};

// A score wave's chunk: y'' of the tokens 16 IT .., in results of spread channels:
// y[2h] and y[2h + 1] hold token lane % 16's channels 32h + 8q .. +3 and +4 .. +7.
template <int SP, int IT>
SEQ_DEV void score_rows(const bf16_t *sC, const bf16_t *sB, const bf16_t *sX, const float *cum, const float *low,
                        const float *dt, float skip, int lane, f32x4 (&y)[4])
{
    typedef Ring<SP> BR;
    typedef Ring<kPB> XR;
    constexpr int KN = SP / 32, KQ = IT / 2 + 1;
    const int q = lane >> 4, l16 = lane & 15, i = IT * 16 + l16;
    bf16x8 cf[KN], bf[2][KN], xf[KQ][4];
    f32x4 s[2 * KQ];
    auto read_b = [&](int jt) __attribute__((always_inline)) {
#pragma unroll
        for (int ks = 0; ks < KN; ++ks) bf[jt & 1][ks] = BR::rows(sB, jt * 16, ks * 32, lane);
    };
#pragma unroll
    for (int ks = 0; ks < KN; ++ks) cf[ks] = BR::rows(sC, IT * 16, ks * 32, lane);
    read_b(0);
    const float ci = cum[i], li = low[i];
    f32x4 ex[IT + 1], dj[IT + 1];
#pragma unroll
    for (int jt = 0; jt <= IT; ++jt) {
        ex[jt] = (ci - *reinterpret_cast<const f32x4 *>(cum + jt * 16 + q * 4)) +
                 (li - *reinterpret_cast<const f32x4 *>(low + jt * 16 + q * 4));
        dj[jt] = *reinterpret_cast<const f32x4 *>(dt + jt * 16 + q * 4);
    }
#pragma unroll
    for (int jt = 0; jt < 2 * KQ; ++jt) s[jt] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int jt = 0; jt <= IT; ++jt) {
        if (jt < IT) {
            read_b(jt + 1);
        } else {
#pragma unroll
            for (int ks = 0; ks < KQ; ++ks)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    xf[ks][2 * h] = XR::template cols<true, 0>(sX, ks * 32, h * 32, lane);
                    xf[ks][2 * h + 1] = XR::template cols<true, 1>(sX, ks * 32, h * 32, lane);
                }
        }
        in_order();
        // the decays of the tile before go with the products of this one
        if (jt > 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) s[jt - 1][r] *= exp2_fast(ex[jt - 1][r]) * dj[jt - 1][r];
        }
#pragma unroll
        for (int ks = 0; ks < KN; ++ks) s[jt] = mma(bf[jt & 1][ks], cf[ks], s[jt]);
        in_order();
    }
    // the tile on the diagonal, with D there
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        s[IT][r] = l16 >= q * 4 + r ? s[IT][r] * exp2_fast(ex[IT][r]) * dj[IT][r] : 0.0f;
        if (l16 == q * 4 + r) s[IT][r] += skip;
    }
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) y[pt] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int ks = 0; ks < KQ; ++ks) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = s[2 * ks][e], v[4 + e] = s[2 * ks + 1][e];
        Split<bf16_t, 3> ms;
        make_split(v, ms);
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
            for (int pt = 0; pt < 4; ++pt) y[pt] = mma(xf[ks][pt], ms.f[m], y[pt]);
    }
}

template <int SP> __global__ void __launch_bounds__(512) scan_fwd_dma_kernel(ScanParams p)
{
    constexpr int Q = 64, NT = SP / 16, KN = SP / 32, STAGE = FwdDmaShared<SP>::STAGE;
    typedef Ring<kPB> XR;
    typedef Ring<SP> BR;
    constexpr int LOADS = 2 * BR::LOADS + XR::LOADS;
    static_assert(LOADS < 64, "all of a chunk's loads fit the counter");
    __shared__ FwdDmaShared<SP> sh;
    const int lane = threadIdx.x & 63, w = wave_id(), q = lane >> 4, l16 = lane & 15;
    const int nseg = p.nseg / p.sub;
    const int64_t unit = blockIdx.x / nseg;
    const int seg = (int)(blockIdx.x - unit * nseg);
    const int pb = (int)(unit % p.NPB);
    const int64_t nh = unit / p.NPB, n = nh / p.H;
    const int h = (int)(nh - n * p.H), g = h / (p.H / p.G);
    const int64_t len = seq_len(p.lengths, n, p.L);
    const int pcols = min(kPB, p.P - pb * kPB);
    const bf16_t *xg = (const bf16_t *)p.x + n * p.L * p.x_ld + (int64_t)h * p.P + pb * kPB;
    const bf16_t *bg = (const bf16_t *)p.b + n * p.L * p.b_ld + (int64_t)g * p.S;
    const bf16_t *cg = (const bf16_t *)p.c + n * p.L * p.c_ld + (int64_t)g * p.S;
    const bf16_t *dg = (const bf16_t *)p.dt + n * p.L * p.dt_ld + h;
    bf16_t *yg = (bf16_t *)p.y + n * p.L * p.y_ld + (int64_t)h * p.P + pb * kPB;
    const float a = p.a[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f, skip = p.d ? p.d[h] : 0.0f;
    const int c_lo = seg * p.seg * p.sub, c_hi = min(p.K, c_lo + p.seg * p.sub);
    const int c_live = (int)min((int64_t)c_hi, (len + Q - 1) / Q);
    const int steps = max(0, c_live - c_lo);
    const int ch = w * 16 + l16;                // a state wave's channel
    const bool busy = w * 16 < pcols;           // a state wave with channels

    float raw = 0.0f;
    auto fetch_dt = [&](int k) __attribute__((always_inline)) {
        const int64_t t = (int64_t)(c_lo + k) * Q + lane;
        raw = k < steps && t < len ? (float)dg[t * p.dt_ld] + bias : 0.0f;
    };
    // The decays of chunk k, a long chain of scalar work, into slot k % 3: two
    // score waves do those of the next two chunks at every second one.
    auto decays = [&](int k, int to) __attribute__((always_inline)) {
        float dt;
        double cum;
        chunk_decay(raw, k < steps && (int64_t)(c_lo + k) * Q + lane < len, a, p.softplus, dt, cum);
        const double tot = wave_last(cum);
        sh.cum[to][lane] = (float)cum;
        sh.low[to][lane] = (float)(cum - (double)(float)cum);
        sh.dt[to][lane] = dt;
        sh.w[to][lane] = exp2_fast((float)(tot - cum)) * dt;
    };
    int stage = 0, slot = 0;        // where a chunk and its decays are
    // wave 4's part of the ring: load g of a tile takes rows one row on from load g - 1
    const uint32_t ring = lds_address(sh.ring);
    int fill = 0;
    auto issue = [&](int k) __attribute__((always_inline)) {
        const int64_t t0 = (int64_t)(c_lo + k) * Q;
        const int rows = (int)min((int64_t)Q, len - t0);
        const i32x4_t xb = chunk_buffer(xg + t0 * p.x_ld, p.x_ld, rows, pcols);
        const i32x4_t bb = chunk_buffer(bg + t0 * p.b_ld, p.b_ld, rows, p.S);
        const i32x4_t cb = chunk_buffer(cg + t0 * p.c_ld, p.c_ld, rows, p.S);
        uint32_t to = ring + fill, from = BR::source(0, lane, (int)p.c_ld, p.S);
#pragma unroll
        for (int g = 0; g < BR::LOADS; ++g, to += 2 * BR::GROUP, from += 2 * (uint32_t)p.c_ld) dma16(cb, from, 0, to);
        from = BR::source(0, lane, (int)p.b_ld, p.S);
#pragma unroll
        for (int g = 0; g < BR::LOADS; ++g, to += 2 * BR::GROUP, from += 2 * (uint32_t)p.b_ld) dma16(bb, from, 0, to);
        from = XR::source(0, lane, (int)p.x_ld, pcols);
#pragma unroll
        for (int g = 0; g < XR::LOADS; ++g, to += 2 * XR::GROUP, from += 2 * (uint32_t)p.x_ld) dma16(xb, from, 0, to);
        fill = next_stage(fill, STAGE);
    };
    if (w < 4) {
        f32x4 st[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) st[t] = f32x4{0, 0, 0, 0};
        if (p.state && ch < pcols) {
            const float *s = p.state + (nh * p.P + pb * kPB + ch) * p.S;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (spread_state(t, q, r) < p.S) st[t][r] = s[spread_state(t, q, r)];
        }
        join_segments<SP, false>(p, unit, seg * p.sub, st, [&](const float *v, int t) __attribute__((always_inline)) {
            return *reinterpret_cast<const f32x4 *>(v + ch * SP + spread_state(t, q, 0));
        });
        if (steps > 0) __syncthreads();
        const int lane_ = lane;
        for (int k = 0; k < steps; ++k) {
            const int lane = fresh_vector(lane_), q = lane >> 4, l16 = lane & 15;      // as in scan_bwd_kernel
            const bf16_t *sC = (const bf16_t *)(sh.ring + stage), *sB = sC + BR::BYTES / 2, *sX = sB + BR::BYTES / 2;
            const float *cum = sh.cum[slot], *wt = sh.w[slot];
            stage = next_stage(stage, STAGE);
            slot = slot == 2 ? 0 : slot + 1;
            if (busy) {
                bf16x8 cf[KN][4], xf[2], bf[NT];
                f32x4 y[4], w0[2], w1[2];
                float ei[4];
                Split<bf16_t, 3> hs[2];
                Split<bf16_t, 3> xs[2];
                auto read_b = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
                    for (int t = 0; t < NT; t += 2) {
                        bf[t] = BR::template cols<true, 0>(sB, ks * 32, t * 16, lane);
                        bf[t + 1] = BR::template cols<true, 1>(sB, ks * 32, t * 16, lane);
                    }
                };
                auto split_h = [&](int ks) __attribute__((always_inline)) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = st[2 * ks][e], v[4 + e] = st[2 * ks + 1][e];
                    make_split(v, hs[ks & 1]);
                };
                auto split_x = [&](int ks) __attribute__((always_inline)) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = (float)xf[ks][e] * (e < 4 ? w0[ks][e & 3] : w1[ks][e & 3]);
                    make_split(v, xs[ks]);
                };
#pragma unroll
                for (int ks = 0; ks < KN; ++ks)
#pragma unroll
                    for (int it = 0; it < 4; ++it) cf[ks][it] = BR::rows(sC, it * 16, ks * 32, lane);
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    xf[ks] = XR::cols(sX, ks * 32, w * 16, lane);
                    w0[ks] = *reinterpret_cast<const f32x4 *>(wt + ks * 32 + q * 4);
                    w1[ks] = *reinterpret_cast<const f32x4 *>(wt + ks * 32 + 16 + q * 4);
                }
#pragma unroll
                for (int it = 0; it < 4; ++it) ei[it] = cum[it * 16 + l16];
                const float dec = exp2_fast(cum[Q - 1]);
                in_order();
#pragma unroll
                for (int it = 0; it < 4; ++it) y[it] = f32x4{0, 0, 0, 0};
                split_h(0);
                // the splits of the next operands go with the products
#pragma unroll
                for (int ks = 0; ks < KN; ++ks) {
                    if (ks + 1 < KN) {
                        split_h(ks + 1);
                    } else {
                        split_x(0);
#pragma unroll
                        for (int t = 0; t < NT; ++t) st[t] *= dec;
                    }
                    if (ks == (KN > 1 ? KN - 2 : 0)) read_b(0);
#pragma unroll
                    for (int m = 0; m < 3; ++m)
#pragma unroll
                        for (int it = 0; it < 4; ++it) y[it] = mma(hs[ks & 1].f[m], cf[ks][it], y[it]);
                    in_order();
                }
                split_x(1);
#pragma unroll
                for (int m = 0; m < 3; ++m)
#pragma unroll
                    for (int t = 0; t < NT; ++t) st[t] = mma(bf[t], xs[0].f[m], st[t]);
                in_order();
                read_b(1);
                in_order();
                // y' goes to the score waves
#pragma unroll
                for (int it = 0; it < 4; ++it)
                    *reinterpret_cast<f32x4 *>(&sh.y[k & 1][(it * 16 + l16) * kPB + (((w * 4 + q) ^ l16) << 2)]) =
                        y[it] * exp2_fast(ei[it]);
#pragma unroll
                for (int m = 0; m < 3; ++m)
#pragma unroll
                    for (int t = 0; t < NT; ++t) st[t] = mma(bf[t], xs[1].f[m], st[t]);
            }
            __syncthreads();
        }
        if (p.state_out && seg == nseg - 1 && ch < pcols) {
            float *s = p.state_out + (nh * p.P + pb * kPB + ch) * p.S;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (spread_state(t, q, r) < p.S) s[spread_state(t, q, r)] = st[t][r];
        }
    } else {
        const int it = w - 4;
        f32x4 y[4];
        // rows behind the sequence come out as zeros, whatever the state times zero is
        auto finish = [&](int k, int lane) __attribute__((always_inline)) {
            const int q = lane >> 4, l16 = lane & 15, i = it * 16 + l16;
            const int64_t t0 = (int64_t)(c_lo + k) * Q;
            const int rows = (int)min((int64_t)Q, p.L - t0);
            const __amdgpu_buffer_rsrc_t buf = __builtin_amdgcn_make_buffer_rsrc(
                yg + t0 * p.y_ld, 0, (int)(((rows - 1) * p.y_ld + pcols) * 2), 0x00020000);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = h * 32 + q * 8;
                if (h * 32 >= pcols) continue;
                bf16x8 o;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int piece = h * 8 + q * 2 + m;
                    const float *from = &sh.y[k & 1][i * kPB + ((piece ^ l16) << 2)];
                    const f32x4 v = y[2 * h + m] + *reinterpret_cast<const f32x4 *>(from);
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[m * 4 + r] = (bf16_t)v[r];
                }
                if (t0 + i >= len) o = bf16x8{0, 0, 0, 0, 0, 0, 0, 0};
                const uint32_t to = col < pcols ? (uint32_t)(i * (int)p.y_ld + col) * 2 : kOutOfRange;
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), buf, to, 0, kStream);
            }
        };
        const bool decaying = it == 1 || it == 2;
        if (steps > 0) {
            if (decaying) {
                fetch_dt(it - 1);
                decays(it - 1, it - 1);
                fetch_dt(it + 1);
            }
            if (it == 0) {
                issue(0);
                if (steps > 1) {
                    issue(1);
                    wait_vmcnt<LOADS>();
                } else {
                    wait_vmcnt<0>();
                }
            }
            __syncthreads();
        }
        const int lane_ = lane;
        for (int k = 0; k < steps; ++k) {
            const int lane = fresh_vector(lane_);      // as in scan_bwd_kernel
            if (k > 0) finish(k - 1, lane);
            if (it == 0 && k + 2 < steps) issue(k + 2);       // over chunk k - 1, which all waves are done with
            const bf16_t *sC = (const bf16_t *)(sh.ring + stage), *sB = sC + BR::BYTES / 2, *sX = sB + BR::BYTES / 2;
            const float *cum = sh.cum[slot], *low = sh.low[slot], *dt = sh.dt[slot];
            stage = next_stage(stage, STAGE);
            slot = slot == 2 ? 0 : slot + 1;
            if (it == 0) score_rows<SP, 0>(sC, sB, sX, cum, low, dt, skip, lane, y);
            else if (it == 1) score_rows<SP, 1>(sC, sB, sX, cum, low, dt, skip, lane, y);
            else if (it == 2) score_rows<SP, 2>(sC, sB, sX, cum, low, dt, skip, lane, y);
            else score_rows<SP, 3>(sC, sB, sX, cum, low, dt, skip, lane, y);
            if ((k & 1) && decaying) {      // chunks k + 1 and k + 2: the slots that are neither k's
                decays(k + it, it == 1 ? slot : slot == 2 ? 0 : slot + 1);
                fetch_dt(k + 2 + it);
            }
            if (it == 0) {      // all but chunk k + 2's have arrived
                if (k + 2 < steps) wait_vmcnt<LOADS>();
                else wait_vmcnt<0>();
            }
            __syncthreads();
        }
        if (steps > 0) finish(steps - 1, lane);
        // chunks behind the sequence: zeros
        for (int c = max(c_lo, c_live); c < c_hi; ++c)
            for (int e = threadIdx.x - 256; e < Q * kPB / 8; e += 256) {
                const int64_t t = (int64_t)c * Q + e / (kPB / 8);
                const int col = e % (kPB / 8) * 8;
                if (t < p.L && col < pcols) *reinterpret_cast<u32x4 *>(yg + t * p.y_ld + col) = u32x4{0, 0, 0, 0};
            }
    }
}

}  // namespace convfwd
