// w4.hip -- the experts' products for few tokens, with weights in 4 bits.
//
// While text is generated a step routes a handful of tokens: each expert
// that is chosen multiplies its two matrices by a few vectors, so the time is
// the chosen weights' bytes. They are held as OCP MXFP4 (Microscaling v1.0):
// per 32 elements of a row one E8M0 scale, and elements of one sign, two
// exponent and one mantissa bit (0, 1/2, 1, 3/2, 2, 3, 4, 6), two a byte, the
// first in the low half: 17/32 of a byte a weight.
//
//   a_r, b_r = W1[e] x[token of row r]   h_r = silu(a_r) b_r   y_r = W2[e] h_r
//   out[t] = sum_j g[t, j] y[token_pos[t, j]]
//
// A wave multiplies 16 rows of weights by up to 16 columns with
// v_mfma_f32_16x16x32_bf16: the four-bit elements are widened to bf16, which
// holds them exactly with their scale (v_cvt_scalef32_pk_bf16_fp4), one
// scale block of 32 per lane. Which 8 of the 32 reduction indices a lane
// brings is free as long as both operands agree: here lane l takes block
// 4 s + l / 16 of row l % 16 in step s, 16 contiguous bytes, in four MFMAs,
// so weights are kept in their plain layout. h is handed on as the sum of two
// bf16 (16 significant bits, each in columns of its own) and y in fp32: the
// only rounding to bf16 is out's.
//
// Bound by the weights' bytes with tokens for most experts, by the latency of
// a launch and a chain of loads with few. d = 2048, h = 1024, E = 128, k = 4: 64
// tokens (111 experts, 371 MB) 48 + 28 + 5 us, 4.6 TB/s of the 6.1 that a plain
// read of memory reaches; one token (4 experts, 13 MB) 6.1 + 5.9 us. What it took
// (gate and up, down at 64 tokens): no branch around a load (106 -> 77, ..),
// memory read by runs of lanes and put into the product's order through LDS
// (77 -> 58: the first-level cache looked up 39 million lines for the 4 million
// there are), tokens no more than 8 at a time (.., 47 -> 34: registers and LDS
// for 16 leave a third of the waves out), the scale bytes of two steps in one
// load, weights asked for before the rows' tokens are known (53 -> 51, 34 ->
// 32), half as many workgroups (51 -> 49, 32 -> 31), runs of whole cache lines
// (49 -> 47), h's halves side by side in one product and LDS rows an odd number
// of pieces apart, whose places are constants and not registers (.., 31 -> 28).
// The loads alone, in the same order, take 44 and 25. Slower were loads past the last-level cache, whole rows a wave, the next
// step's weights in flight during a step (59 and 33 us one step at a time, no
// gain and spilled registers two at a time), twice the registers for loads,
// more waves with fewer loads each (55 and 37 us).
#include "act8.h"

namespace moe {

// ---------------------------------------------------------------------------
// quantisation: thread = 8 elements, 4 lanes a block of 32. Bound by memory: 128
// experts of d = 2048, h = 1024 from fp32 635 us for 3.65 GB (5.7 TB/s), from bf16
// 331 us for 2.04 GB (6.2 TB/s).

template <bool BF16>
__global__ __launch_bounds__(256) void w4_quantize_vecs(const uint4 *__restrict__ in, int64_t n8,
                                                        uint32_t *__restrict__ q,
                                                        uint8_t *__restrict__ scale) {
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n8) return;                          // whole blocks: n8 % 4 == 0
    float f[8];
    if constexpr (BF16)
        Row16<true>::unpack(in[v], f);
    else {
        Row16<false>::unpack(in[2 * v], f);
        Row16<false>::unpack(in[2 * v + 1], f + 4);
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) amax = fmaxf(amax, fabsf(f[i]));
    amax = fmaxf(amax, dpp_move<kDppXor1>(amax));
    amax = fmaxf(amax, dpp_move<kDppXor2>(amax));
    // floor(log2 amax) - 2: the largest element, 6, is 3/2 * 2^2
    const uint32_t sb = (uint32_t)max((int)((__float_as_uint(amax) >> 23) & 0xff) - 2, 0);
    const float s = __uint_as_float(sb << 23);    // the instruction reads the exponent field
    const float top = ldexpf(6.f, (int)sb - 127);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = __builtin_amdgcn_fmed3f(f[i], -top, top);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], s, 3);
    q[v] = w;
    if ((v & 3) == 0) scale[v >> 2] = (uint8_t)sb;
}

// ---------------------------------------------------------------------------
// the products

// eight four-bit elements to bf16, scaled
MOE_DEV bf16x8 w4_widen(uint32_t w, float s) {
    const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    const bf16x8 r = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    return r;
}

// The expert with rank `slot` among those with rows, and its rows; false if
// there are fewer. Every wave finds it by itself: expert 64 i + lane in turn.
MOE_DEV bool w4_active(const int32_t *offsets, int E, int slot, int &e, int &r0, int &r1) {
    const int lane = threadIdx.x & 63;
    int a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int x = 64 * i + lane;
        a[i] = x < E ? offsets[x] : 0;
        b[i] = x < E ? offsets[x + 1] : 0;
    }
    int before = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint64_t m = __ballot(b[i] > a[i]);
        const int n = __popcll(m);
        if (!found && slot < before + n) {           // uniform
            const int rank = before + __popcll(m & (((uint64_t)1 << lane) - 1));
            const int l = __ffsll(__ballot(b[i] > a[i] && rank == slot)) - 1;
            e = 64 * i + l;
            r0 = __builtin_amdgcn_readlane(a[i], l);
            r1 = __builtin_amdgcn_readlane(b[i], l);
            found = true;
        }
        before += n;
    }
    return found;
}

constexpr int kW4Tokens = 8;     // rows of an expert that a wave multiplies at once
constexpr int kW4Steps = 2;      // steps of 128 reduction indices loaded at once
constexpr int kW4WideTiles = 2;  // row tiles of 16 with many rows
constexpr int kW4WideSteps(bool up) { return up ? 4 : 2; }    // steps of a piece

struct W4Args {
    const uint16_t *x;           // UP: x [T, d]; else h's upper halves [R, h]
    const uint16_t *lo;          // down: h's lower halves [R, h]
    const int32_t *sorted_token; // UP: token of a row
    const uint8_t *wq, *ws;
    uint16_t *hi_out, *lo_out;   // UP: h
    float *y;                    // down: y [R, d]
    int K, h, d;
};

// The two tiles of 16 weight rows that a wave multiplies (the same for all of
// its lanes, so that the lanes need offsets of 32 bits alone).
struct W4Tiles {
    const uint8_t *q0, *q1, *s0, *s1;
    MOE_DEV W4Tiles(const W4Args &p, int64_t row0, int64_t row1) {
        const int nblk = p.K / 32;
        q0 = p.wq + row0 * 16 * nblk; q1 = p.wq + row1 * 16 * nblk;
        s0 = p.ws + row0 * nblk; s1 = p.ws + row1 * nblk;
    }
};

MOE_DEV int w4_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// U bytes
template <int U> struct W4Bytes;
template <> struct W4Bytes<1> { typedef uint8_t type; };
template <> struct W4Bytes<2> { typedef uint16_t type; };
template <> struct W4Bytes<4> { typedef uint32_t type; };

// What a wave keeps in LDS: both weight tiles of the U steps that were loaded
// together (16 rows of 4 U blocks, 16 bytes each) with their scales, and of one
// step TOK tokens (their upper halves, then their lower ones, of h) of 4 blocks
// in 16-byte pieces.
template <bool UP, int TOK, int U>
struct W4Stage {
    u32x4 w[2][16 * (4 * U + 1)];
    uint8_t sc[2][64 * U];
    u32x4 x[(UP ? 1 : 2) * TOK * 17];
};

// Rows are one piece apart from their length, an odd number, so that the 16
// lanes that read one piece of 16 rows each meet different banks.
template <int U>
MOE_DEV int w4_wslot(int row, int blk) { return (4 * U + 1) * row + blk; }
MOE_DEV int w4_xslot(int row, int piece) { return 17 * row + piece; }

// The lanes of a wave see each other's LDS writes in program order; this
// keeps the compiler to that order.
MOE_DEV void w4_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The weights of steps [s, s + U) of a wave's reduction: 4 U blocks of 16 rows
// of each tile, and U scale bytes a lane. Memory is read in contiguous runs, 64
// U bytes of a row by 4 U lanes. TAIL: blocks past the row's end count as zeros.
template <int U, bool TAIL>
struct W4Loaded {
    u32x4 w[U][2];                                // row 16 / U * q + lane / (4 U)
    typename W4Bytes<U>::type sc[2];              // row lane / 4
    MOE_DEV void load(int s, int nblk, const W4Tiles &wt) {
        static_assert(!TAIL || U == 1);
        const int lane = threadIdx.x & 63, lr = lane >> 2, lc = lane & 3;
        const int c = 4 * s + lane % (4 * U);
        const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < U; q++) {
            w[q][0] = w[q][1] = zero;
            if (!TAIL || c < nblk) {
                const uint32_t o = (16 / U * q + lane / (4 * U)) * nblk + c;     // block of the tile
                w[q][0] = *reinterpret_cast<const u32x4 *>(wt.q0 + 16 * o);
                w[q][1] = *reinterpret_cast<const u32x4 *>(wt.q1 + 16 * o);
            }
        }
        // scales: 4 U bytes of a row, U (at any address) a lane
        sc[0] = sc[1] = 127;
        if (!TAIL || 4 * s + lc < nblk) {
            const uint32_t o = lr * nblk + 4 * s + U * lc;
            __builtin_memcpy(&sc[0], wt.s0 + o, U);
            __builtin_memcpy(&sc[1], wt.s1 + o, U);
        }
    }
};

// Their products: the tokens' loads (16 lanes 256 bytes of token 4 j + lane /
// 16, at x[j] and, of h, its lower half lo elements on, for j < quads; both are
// uniform), then through LDS to the
// matrix units, which want row lane % 16 (a load in the product's own order has
// a lane per row and costs the first-level cache many times the accesses). TOK
// tokens fill the product's 16 columns over and over; of h, the upper halves
// columns 0 to 7 and the lower ones columns 8 to 15, whose sum is the result.
template <bool UP, int TOK, int U, int SU, bool TAIL>
MOE_DEV void w4_steps(int s, int nblk, const W4Loaded<U, TAIL> &l, int quads,
                      const uint16_t *const (&x)[(TOK + 3) / 4], int64_t lo, W4Stage<UP, TOK, SU> &st,
                      f32x4 (&acc)[2]) {
    constexpr int P = UP ? 1 : 2, J = (TOK + 3) / 4;    // h comes as two halves
    typedef typename W4Bytes<U>::type Sc;
    static_assert(UP || TOK <= 8);
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
    const int column = (i & (TOK - 1)) + (UP ? 0 : i / 8 * TOK);
    const u32x4 zero = {0, 0, 0, 0};
    u32x4 xr[U][P][J];
#pragma unroll
    for (int j = 0; j < J; j++)
        if (j == 0 || j < quads) {
#pragma unroll
            for (int p = 0; p < P; p++)
#pragma unroll
                for (int u = 0; u < U; u++)
                    xr[u][p][j] = !TAIL || 4 * (s + u) + (i >> 2) < nblk
                        ? *reinterpret_cast<const u32x4 *>(x[j] + p * lo + 128 * (s + u) + 8 * i) : zero;
        }
    w4_lds_order();                               // the steps before have been read
#pragma unroll
    for (int z = 0; z < 2; z++) {
#pragma unroll
        for (int q = 0; q < U; q++)
            st.w[z][w4_wslot<U>(16 / U * q + lane / (4 * U), lane % (4 * U))] = l.w[q][z];
        *reinterpret_cast<Sc *>(&st.sc[z][U * lane]) = l.sc[z];
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        if (u) w4_lds_order();                    // the step before has been read
#pragma unroll
        for (int j = 0; j < J; j++)
            if (j == 0 || j < quads) {
#pragma unroll
                for (int p = 0; p < P; p++)
                    if (TOK >= 4 || g == 0) st.x[w4_xslot(p * TOK + 4 * j + g, i)] = xr[u][p][j];
            }
        w4_lds_order();
        u32x4 a[2];
        float f[2];
#pragma unroll
        for (int z = 0; z < 2; z++) {
            a[z] = st.w[z][w4_wslot<U>(i, 4 * u + g)];
            f[z] = __uint_as_float((uint32_t)st.sc[z][4 * (U * i + u) + g] << 23);
        }
#pragma unroll
        for (int m = 0; m < 4; m++) {
            const bf16x8 a0 = w4_widen(a[0][m], f[0]), a1 = w4_widen(a[1][m], f[1]);
            const bf16x8 b = __builtin_bit_cast(bf16x8, st.x[w4_xslot(column, 4 * g + m)]);
            acc[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, b, acc[0], 0, 0, 0);
            acc[1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, b, acc[1], 0, 0, 0);
        }
    }
}

// Steps [s, end) of a wave, U at a time. address(): forms x, after the first
// weights have been asked for.
template <bool UP, int TOK, int U, class Address>
MOE_DEV void w4_reduce(int s, int end, int nblk, const W4Tiles &wt, int quads, Address address,
                       int64_t lo, W4Stage<UP, TOK, U> &st, f32x4 (&acc)[2]) {
    const uint16_t *x[(TOK + 3) / 4];
    const int whole = min(end, nblk / 4);
    W4Loaded<U, false> l;
    const bool any = s + U <= whole;
    if (any) l.load(s, nblk, wt);
    address(x);
    if (any)
        for (;;) {
            w4_steps<UP, TOK>(s, nblk, l, quads, x, lo, st, acc);
            s += U;
            if (s + U > whole) break;
            l.load(s, nblk, wt);
        }
    for (; s < end; s++) {
        W4Loaded<1, true> t;
        t.load(s, nblk, wt);
        w4_steps<UP, TOK>(s, nblk, t, quads, x, lo, st, acc);
    }
}

// LDS of a workgroup: the waves' stages, then their sums.
template <bool UP, int TOK, int U>
union W4Lds {
    W4Stage<UP, TOK, U> stage[4];
    float red[4][2][256];
};

// N results of row `row`, columns from n: h as its two halves, or y. The upper
// half of an h beyond bf16's largest value (0x7f7f) is that value, so that the
// rest is finite where h is and the infinity where h is infinite.
template <bool UP, int N>
MOE_DEV void w4_store(const W4Args &p, int64_t row, int n, const float *v0, const float *v1) {
    if constexpr (UP) {
        uint16_t hi[N], lo[N];
#pragma unroll
        for (int q = 0; q < N; q++) {
            const float o = silu(v0[q]) * v1[q];
            const float top = bf16_to_f32(0x7f7f);
            hi[q] = f32_to_bf16(__builtin_amdgcn_fmed3f(o, -top, top));
            lo[q] = f32_to_bf16(o - bf16_to_f32(hi[q]));
        }
        __builtin_memcpy(p.hi_out + row * p.h + n, hi, sizeof(hi));
        __builtin_memcpy(p.lo_out + row * p.h + n, lo, sizeof(lo));
    } else {
        __builtin_memcpy(p.y + row * p.d + n, v0, N * sizeof(float));
        __builtin_memcpy(p.y + row * p.d + n + 16, v1, N * sizeof(float));
    }
}

// Rows [r, r + TOK) of the expert's rows [.., r1). KS waves share the two
// tiles of 16 weight rows (gate and up of 16 columns, or 32 rows of W2), a
// part of the reduction each, and join their sums in LDS; 4 / KS such pairs
// side by side, from column n0 of n. The columns of the product past the
// expert's last row repeat it, or hold what LDS held (a token is a column: it
// reaches no other), and are not stored.
template <bool UP, int TOK, int U, int KS>
MOE_DEV void w4_rows(const W4Args &p, const W4Tiles &wt, int n0, int n, int r, int r1,
                     W4Lds<UP, TOK, U> &lds) {
    const int lane = threadIdx.x & 63, wave = w4_wave(), g = lane >> 4, i = lane & 15;
    const int nblk = p.K / 32;
    auto address = [&](const uint16_t *(&x)[TOK / 4]) {
#pragma unroll
        for (int j = 0; j < TOK / 4; j++) {
            const int row = min(r + 4 * j + g, r1 - 1);
            x[j] = p.x + (UP ? p.sorted_token[row] : row) * (int64_t)p.K;
        }
    };
    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    const int steps = (nblk + 3) / 4, part = (steps + KS - 1) / KS, s = (wave % KS) * part;
    w4_reduce<UP, TOK, U>(s, min(s + part, steps), nblk, wt, (r1 - r + 3) / 4, address,
                          UP ? 0 : p.lo - p.x, lds.stage[wave], acc);
    // lane: column i (token i while i < TOK), weight rows 4 g .. 4 g + 3
    __syncthreads();                              // the stages have been read
#pragma unroll
    for (int z = 0; z < 2; z++) *reinterpret_cast<f32x4 *>(&lds.red[wave][z][i * 16 + 4 * g]) = acc[z];
    __syncthreads();
    const int tid = threadIdx.x, tok = tid >> 4;
#pragma unroll
    for (int t = 0; t < 4 / KS; t++) {
        float v[2];
#pragma unroll
        for (int z = 0; z < 2; z++) {
            v[z] = 0;
#pragma unroll
            for (int q = 0; q < KS; q++) {
                v[z] += lds.red[t * KS + q][z][tid];
                if (!UP) v[z] += lds.red[t * KS + q][z][(tid + 128) & 255];
            }
        }
        const int n1 = n0 + t * (UP ? 16 : 32);
        if (tok < TOK && r + tok < r1 && n1 < n) w4_store<UP, 1>(p, r + tok, n1 + (tid & 15), &v[0], &v[1]);
    }
    __syncthreads();                              // the sums have been read
}

// An expert's rows are shared out to Z workgroups for each group of columns;
// those Z are 8 apart, so that they run on one XCD and its cache serves the
// weights again.
MOE_DEV void w4_place(int Z, int &col, int &z) {
    const int x = blockIdx.x;
    col = Z == 1 ? x : x / (8 * Z) * 8 + x % 8;
    z = Z == 1 ? 0 : x / 8 % Z;
}
static unsigned w4_grid(int cols, int Z) { return Z == 1 ? cols : (cols + 7) / 8 * 8 * Z; }

// column group: 16 columns of h (UP) or 32 of d, times 4 / KS; blockIdx.y: rank
// of an expert with rows
template <bool UP, int KS>
__global__ __launch_bounds__(256, 4) void w4_product(W4Args p, const int32_t *__restrict__ offsets,
                                                     int E, int Z) {
    __shared__ W4Lds<UP, kW4Tokens, kW4Steps> lds;
    int e, r0, r1;
    if (!w4_active(offsets, E, blockIdx.y, e, r0, r1)) return;      // the whole workgroup
    constexpr int C = UP ? 16 : 32;
    int col, z;
    w4_place(Z, col, z);
    const int n = UP ? p.h : p.d, n0 = col * C * (4 / KS);
    if (n0 >= n) return;
    // waves past the last column multiply it again and store nothing
    const int m0 = min(n0 + w4_wave() / KS * C, n - C);
    const int64_t w0 = (int64_t)e * (UP ? 2 * p.h : p.d) + m0;
    const W4Tiles wt(p, w0, w0 + (UP ? p.h : 16));
    for (int r = r0 + z * kW4Tokens; r < r1; r += Z * kW4Tokens)
        w4_rows<UP, kW4Tokens, kW4Steps, KS>(p, wt, n0, n, r, r1, lds);
}

// Many rows an expert: rows [r, r + 16 NT), every wave its own two tiles of
// weight rows over the whole reduction, in pieces of PS steps. The workgroup
// keeps a piece of its tokens in LDS for all four waves, a wave two steps of its
// weights; the next piece, tokens and weights, is in flight while one is
// computed.
template <bool UP, int NT, int PS>
struct W4Wide {
    u32x4 x[UP ? 1 : 2][NT][16 * (16 * PS + 1)];  // 16 tokens of 16 PS pieces of 16 bytes
    u32x4 w[4][2][16 * 9];
    uint8_t sc[4][2][16 * 4 * PS];
};

// A wave's weights of a piece. Blocks past the row's end repeat its last one
// (no branch around a load), with scale byte 0; they meet tokens that are zero
// there. It is the tokens that have to be: they may hold infinities.
template <int PS>
struct W4Piece {
    u32x4 w[PS / 2][2][2];                        // row 8 q + lane / 8
    typename W4Bytes<PS>::type sc[2];             // row lane / 4, PS bytes
    MOE_DEV void load(int piece, int nblk, const W4Tiles &wt) {
        const int lane = threadIdx.x & 63;
        const uint32_t os = (lane >> 2) * nblk + min(4 * PS * piece + PS * (lane & 3), nblk - PS);
        __builtin_memcpy(&sc[0], wt.s0 + os, PS);
        __builtin_memcpy(&sc[1], wt.s1 + os, PS);
#pragma unroll
        for (int v = 0; v < PS / 2; v++)
#pragma unroll
            for (int q = 0; q < 2; q++) {
                const int c = min(4 * PS * piece + 8 * v + (lane & 7), nblk - 1);
                const uint32_t o = (8 * q + (lane >> 3)) * nblk + c;
                w[v][q][0] = *reinterpret_cast<const u32x4 *>(wt.q0 + 16 * o);
                w[v][q][1] = *reinterpret_cast<const u32x4 *>(wt.q1 + 16 * o);
            }
    }
};

template <bool UP, int NT, int PS>
MOE_DEV void w4_rows_wide(const W4Args &p, const W4Tiles &wt, int n0, bool store, int r, int r1,
                          W4Wide<UP, NT, PS> &lds) {
    constexpr int P = UP ? 1 : 2;
    const int tid = threadIdx.x, lane = tid & 63, wave = w4_wave(), g = lane >> 4, i = lane & 15;
    const int xt = tid >> 4, xc = tid & 15;
    const int nblk = p.K / 32, pieces = (nblk + 4 * PS - 1) / (4 * PS);
    const int tiles = (r1 - r + 15) / 16;         // of tokens; uniform
    const int64_t lo = UP ? 0 : p.lo - p.x;
    const uint16_t *x[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int row = min(r + 16 * t + xt, r1 - 1);
        x[t] = p.x + (UP ? p.sorted_token[row] : row) * (int64_t)p.K;
    }
    const u32x4 zero = {0, 0, 0, 0};
    u32x4 xr[P][NT][PS];
    auto load_x = [&](int piece) {
#pragma unroll
        for (int t = 0; t < NT; t++)
            if (t == 0 || t < tiles) {
#pragma unroll
                for (int q = 0; q < P; q++)
#pragma unroll
                    for (int j = 0; j < PS; j++) {
                        const int c = min(16 * PS * piece + 16 * j + xc, 4 * nblk - 1);
                        xr[q][t][j] = *reinterpret_cast<const u32x4 *>(x[t] + q * lo + 8 * c);
                    }
            }
    };
    f32x4 acc[2][NT];
#pragma unroll
    for (int z = 0; z < 2; z++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[z][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int piece, W4Piece<PS> &now, W4Piece<PS> &next) {
        __syncthreads();                          // the tokens' piece before has been read
#pragma unroll
        for (int t = 0; t < NT; t++)
            if (t == 0 || t < tiles) {
#pragma unroll
                for (int q = 0; q < P; q++)
#pragma unroll
                    for (int j = 0; j < PS; j++)
                        lds.x[q][t][(16 * PS + 1) * xt + 16 * j + xc] =
                            16 * PS * piece + 16 * j + xc < 4 * nblk ? xr[q][t][j] : zero;
            }
        if (piece + 1 < pieces) {
            load_x(piece + 1);
            next.load(piece + 1, nblk, wt);
        }
        __syncthreads();
        const int b0 = 4 * PS * piece;
#pragma unroll
        for (int v = 0; v < PS / 2; v++) {
            w4_lds_order();                       // the steps before have been read
#pragma unroll
            for (int z = 0; z < 2; z++) {
#pragma unroll
                for (int q = 0; q < 2; q++)
                    lds.w[wave][z][9 * (8 * q + (lane >> 3)) + (lane & 7)] = now.w[v][q][z];
                if (v == 0) {
                    const int past = b0 + PS * (lane & 3) - (nblk - PS);     // bytes read too early
                    const uint32_t b = past <= 0 ? now.sc[z] : past < PS ? (uint32_t)now.sc[z] >> (8 * past) : 0;
                    *reinterpret_cast<typename W4Bytes<PS>::type *>(&lds.sc[wave][z][PS * lane]) = b;
                }
            }
            w4_lds_order();
#pragma unroll
            for (int u = 2 * v; u < 2 * v + 2; u++) {
                u32x4 a[2];
                float f[2];
#pragma unroll
                for (int z = 0; z < 2; z++) {
                    a[z] = lds.w[wave][z][9 * i + 4 * (u - 2 * v) + g];
                    f[z] = __uint_as_float((uint32_t)lds.sc[wave][z][4 * (PS * i + u) + g] << 23);
                }
#pragma unroll
                for (int m = 0; m < 4; m++) {
                    const bf16x8 a0 = w4_widen(a[0][m], f[0]), a1 = w4_widen(a[1][m], f[1]);
#pragma unroll
                    for (int t = 0; t < NT; t++)
#pragma unroll
                        for (int q = 0; q < P; q++) {
                            const bf16x8 b = __builtin_bit_cast(
                                bf16x8, lds.x[q][t][(16 * PS + 1) * i + 16 * u + 4 * g + m]);
                            acc[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, b, acc[0][t], 0, 0, 0);
                            acc[1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, b, acc[1][t], 0, 0, 0);
                        }
                }
            }
        }
    };
    W4Piece<PS> even, odd;
    load_x(0);
    even.load(0, nblk, wt);
    for (int piece = 0; piece < pieces; piece += 2) {
        step(piece, even, odd);
        if (piece + 1 < pieces) step(piece + 1, odd, even);
    }
    // lane: token i, weight rows 4 g .. 4 g + 3
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int row = r + 16 * t + i;
        const float v0[4] = {acc[0][t][0], acc[0][t][1], acc[0][t][2], acc[0][t][3]};
        const float v1[4] = {acc[1][t][0], acc[1][t][1], acc[1][t][2], acc[1][t][3]};
        if (store && row < r1) w4_store<UP, 4>(p, row, n0 + 4 * g, v0, v1);
    }
}

// column group: 64 columns of h (UP) or 128 of d, a quarter for each wave;
// blockIdx.y: rank of an expert with rows
template <bool UP, int NT, int PS>
__global__ __launch_bounds__(256, 2) void w4_product_wide(W4Args p,
                                                          const int32_t *__restrict__ offsets,
                                                          int E, int Z) {
    __shared__ W4Wide<UP, NT, PS> lds;
    int e, r0, r1;
    if (!w4_active(offsets, E, blockIdx.y, e, r0, r1)) return;      // the whole workgroup
    int col, z;
    w4_place(Z, col, z);
    const int n0 = (4 * col + w4_wave()) * (UP ? 16 : 32), n = UP ? p.h : p.d;
    if (col * (UP ? 64 : 128) >= n) return;
    // a wave past the last column stages its share of the tokens and stores nothing
    const int m0 = min(n0, n - (UP ? 16 : 32));
    const int64_t w0 = (int64_t)e * (UP ? 2 * p.h : p.d) + m0;
    const W4Tiles wt(p, w0, w0 + (UP ? p.h : 16));
    for (int r = r0 + z * 16 * NT; r < r1; r += Z * 16 * NT) w4_rows_wide<UP, NT, PS>(p, wt, m0, n0 < n, r, r1, lds);
}

// A handful of rows: out[t] for 32 columns from the token's own experts, gates
// and sum included, in one launch (no y, no combine; an expert that tokens
// share is read once for each). Wave: slot wave % 4 and on, half wave / 4 of
// the reduction.
__global__ __launch_bounds__(512, 4) void w4_down_tokens(W4Args p, const int32_t *__restrict__ offsets,
                                                      int E, const float *__restrict__ gate,
                                                      const int32_t *__restrict__ token_pos, int k,
                                                      uint16_t *__restrict__ out) {
    constexpr int U = 4;
    __shared__ W4Stage<false, 1, U> stage[8];
    __shared__ float red[2][8][32], sg[8];
    const int64_t t = blockIdx.y;
    const int lane = threadIdx.x & 63, wave = w4_wave(), g = lane >> 4, i = lane & 15;
    const int n0 = 32 * blockIdx.x, nblk = p.K / 32;
    const int steps = (nblk + 3) / 4, part = (steps + 1) / 2, begin = (wave >> 2) * part;
    const int end = min(begin + part, steps);
    int ends[4];                                  // of the experts' rows
#pragma unroll
    for (int q = 0; q < 4; q++) ends[q] = 64 * q + lane < E ? offsets[64 * q + lane + 1] : INT32_MAX;
    for (int j = wave & 3; j < k; j += 4) {
        const float w = gate[t * k + j];
        const int row = __builtin_amdgcn_readfirstlane(token_pos[t * k + j]);
        f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
        if (row >= 0) {                           // not dropped
            int e = 0;                            // experts that end at or before the row
#pragma unroll
            for (int q = 0; q < 4; q++) e += __popcll(__ballot(ends[q] <= row));
            const W4Tiles wt(p, (int64_t)e * p.d + n0, (int64_t)e * p.d + n0 + 16);
            const int64_t src = (int64_t)row * p.K;
            auto address = [&](const uint16_t *(&x)[1]) { x[0] = p.x + src; };
            w4_reduce<false, 1, U>(begin, end, nblk, wt, 1, address, p.lo - p.x, stage[wave], acc);
        }
#pragma unroll
        for (int z = 0; z < 2; z++)               // columns 0 and 8: the token's halves
#pragma unroll
            for (int q = 0; q < 4; q++) acc[z][q] += dpp_move<kDppRowRor8>(acc[z][q]);
        if (i == 0) {
#pragma unroll
            for (int z = 0; z < 2; z++)
                *reinterpret_cast<f32x4 *>(&red[wave >> 2][j][16 * z + 4 * g]) = acc[z];
            if (lane == 0 && wave < 4) sg[j] = row >= 0 ? w : 0.f;
        }
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
    float v = 0.f;
    for (int j = 0; j < k; j++) v = fmaf(sg[j], red[0][j][threadIdx.x] + red[1][j][threadIdx.x], v);
    out[t * p.d + n0 + threadIdx.x] = f32_to_bf16(v);
}

// out[t] = sum_j g y[token_pos] (fp32, ascending j), 4 columns a thread
__global__ __launch_bounds__(256) void w4_combine(const float *__restrict__ y,
                                                  const float *__restrict__ gate,
                                                  const int32_t *__restrict__ token_pos, int d,
                                                  int k, int cblocks, uint2 *__restrict__ out) {
    const int64_t t = blockIdx.x / cblocks;
    const int c = (blockIdx.x % cblocks) * 256 + threadIdx.x;
    if (4 * c >= d) return;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < k; j++) {
        const int32_t p = token_pos[t * k + j];
        if (p < 0) continue;
        const float g = gate[t * k + j];
        const float4 v = reinterpret_cast<const float4 *>(y + (int64_t)p * d)[c];
        s[0] = fmaf(g, v.x, s[0]); s[1] = fmaf(g, v.y, s[1]);
        s[2] = fmaf(g, v.z, s[2]); s[3] = fmaf(g, v.w, s[3]);
    }
    out[t * (d / 4) + c] = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
}

// ---------------------------------------------------------------------------
// launchers

moe_status w4_quantize_launch(const void *in, moe_dtype dt, int64_t rows, int64_t cols, uint8_t *q,
                              uint8_t *scale, hipStream_t s) {
    const bool bf = dt == MOE_BF16;
    const int64_t n8 = rows * (cols / 8);
    for (int64_t a = 0; a < n8; a += kMaxBlocks * 256) {
        const int64_t n = n8 - a < kMaxBlocks * 256 ? n8 - a : kMaxBlocks * 256;
        const unsigned nb = (unsigned)((n + 255) / 256);
        const uint4 *src = reinterpret_cast<const uint4 *>(in) + a * (bf ? 1 : 2);
        uint32_t *dst = reinterpret_cast<uint32_t *>(q) + a;
        if (bf) w4_quantize_vecs<true><<<nb, 256, 0, s>>>(src, n, dst, scale + a / 4);
        else w4_quantize_vecs<false><<<nb, 256, 0, s>>>(src, n, dst, scale + a / 4);
    }
    return launch_status();
}

static size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// workspace: h's upper halves, its lower halves [R, h] bf16, y [R, d] fp32
size_t w4_ws_bytes(int64_t R, int d, int h) {
    return 2 * round256((size_t)R * h * 2) + round256((size_t)R * d * 4);
}

// One of the two products over n columns. Which kernel, by rows an expert (R /
// E) and workgroups (times of all launches of a call):
//  - from twelve rows an expert, with a workgroup of 64 columns and 32 rows for
//    every compute unit: the wide kernels. d = 2048, h = 1024, E = 128, k = 4, T =
//    512 (16 rows) 134 us against 190; T = 256 (8 rows) 125 both ways; E = 16, k =
//    4, T = 64 (16 rows) 29 against 34, T = 32 27 against 24. E = 8, k = 2, T = 128
//    (128 workgroups) 41 against 30, T = 512 (512) 54 against 79.
//  - five workgroups a compute unit and up: two waves a reduction, not four, so
//    that half as many workgroups look for their expert and join sums. d = 2048,
//    h = 1024, E = 128, k = 4, T = 64 85.3 us against 88.0, E = 256, d = 1024, h =
//    512, k = 8, T = 64 52 against 62; fewer leave compute units out: E = 8, k = 2,
//    T = 16 16.4 against 15.1.
// An expert's rows are shared out to as many workgroups as it takes for four a
// compute unit (eight no better): d = 2048, h = 1024, E = 2, k = 2, T = 256 29 us
// against 135 with one; d = 8192, h = 96, E = 4, k = 2, T = 128 32 against 84.
template <bool UP>
static void w4_product_launch(const moe_w4_desc &w, const W4Args &a, int n, hipStream_t s) {
    const int64_t R = w.T * w.k;
    const unsigned ny = (unsigned)(R < w.E ? R : w.E);
    const int c = n / (UP ? 16 : 32), c2 = (c + 1) / 2, c4 = (c + 3) / 4;
    auto split = [&](int cols, int rows) {
        const int64_t each = (int64_t)rows * ny, parts = (R + each - 1) / each;
        const int64_t z = 1024 / ((int64_t)cols * ny);
        return (int)(z < 1 ? 1 : z < parts ? z : parts);
    };
    const int zw = split(c4, 16 * kW4WideTiles);
    if (R >= 12 * (int64_t)w.E && a.K >= 32 * kW4WideSteps(UP) && (int64_t)c4 * ny * zw >= 256)
        w4_product_wide<UP, kW4WideTiles, kW4WideSteps(UP)><<<dim3(w4_grid(c4, zw), ny), 256, 0, s>>>(a, w.offsets, w.E, zw);
    else if ((int64_t)c * ny >= 1280) {
        const int z = split(c2, kW4Tokens);
        w4_product<UP, 2><<<dim3(w4_grid(c2, z), ny), 256, 0, s>>>(a, w.offsets, w.E, z);
    } else {
        const int z = split(c, kW4Tokens);
        w4_product<UP, 4><<<dim3(w4_grid(c, z), ny), 256, 0, s>>>(a, w.offsets, w.E, z);
    }
}

moe_status w4_experts_launch(const moe_w4_desc *w, hipStream_t s) {
    const int64_t R = w->T * w->k;
    char *ws = reinterpret_cast<char *>(w->ws);
    const size_t half = round256((size_t)R * w->h * 2);
    uint16_t *hi = reinterpret_cast<uint16_t *>(ws), *lo = reinterpret_cast<uint16_t *>(ws + half);
    float *y = reinterpret_cast<float *>(ws + 2 * half);
    const W4Args up = {reinterpret_cast<const uint16_t *>(w->x), nullptr, w->sorted_token, w->w1q,
                       w->w1_scale, hi, lo, nullptr, w->d, w->h, w->d};
    const W4Args down = {hi, lo, nullptr, w->w2q, w->w2_scale, nullptr, nullptr, y, w->h, w->h, w->d};
    const int nd = w->d / 32;
    w4_product_launch<true>(*w, up, w->h, s);
    // A handful of rows: the down product by token (all launches, d = 2048, h =
    // 1024): E = 128, k = 4, T = 8 (R = E / 4) 25.7 us against 28.8; T = 16 (4,096
    // workgroups) 44.9 against 45.0. Where tokens share experts it reads them
    // again: E = 8, k = 2, T = 16 (R = 4 E) 18.8 us against 15.2.
    if (R <= 2 * (int64_t)w->E && nd * R <= 2048) {
        w4_down_tokens<<<dim3(nd, (unsigned)w->T), 512, 0, s>>>(
            down, w->offsets, w->E, w->topk_gate, w->token_pos, w->k,
            reinterpret_cast<uint16_t *>(w->out));
        return launch_status();
    }
    w4_product_launch<false>(*w, down, w->d, s);
    const int cb = (w->d + 1023) / 1024;
    const int64_t piece = kMaxBlocks / cb;
    for (int64_t t = 0; t < w->T; t += piece) {
        const int64_t n = w->T - t < piece ? w->T - t : piece;
        w4_combine<<<(unsigned)(n * cb), 256, 0, s>>>(
            y, w->topk_gate + t * w->k, w->token_pos + t * w->k, w->d, w->k, cb,
            reinterpret_cast<uint2 *>(w->out) + t * (w->d / 4));
    }
    return launch_status();
}

}  // namespace moe
