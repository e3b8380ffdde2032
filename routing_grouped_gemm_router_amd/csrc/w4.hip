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
// A wave multiplies 16 rows of weights by up to 16 tokens with
// v_mfma_f32_16x16x32_bf16: the four-bit elements are widened to bf16, which
// holds them exactly with their scale (v_cvt_scalef32_pk_bf16_fp4), one
// scale block of 32 per lane. Which 8 of the 32 reduction indices a lane
// brings is free as long as both operands agree: here lane l takes block
// 4 s + l / 16 of row l % 16 in step s, 16 contiguous bytes, in four MFMAs,
// so weights are read in their plain layout. h is handed on as the sum of two
// bf16 (16 significant bits) and y in fp32: the only rounding to bf16 is
// out's.
#include "act8.h"

namespace moe {

// ---------------------------------------------------------------------------
// quantisation: thread = 8 elements, 4 lanes a block of 32

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

struct W4Args {
    const uint16_t *x;           // UP: x [T, d]; else h's upper halves [R, h]
    const uint16_t *lo;          // down: h's lower halves [R, h]
    const int32_t *sorted_token; // UP: token of a row
    const uint8_t *wq, *ws;
    uint16_t *hi_out, *lo_out;   // UP: h
    float *y;                    // down: y [R, d]
    int K, h, d;
};

// What a wave keeps in LDS of one step: both weight tiles (16 rows of 4
// blocks, 16 bytes each), their scales, and per row tile (and half of h) 16
// tokens of 4 blocks in 16-byte pieces.
template <bool UP, int NT>
struct W4Stage {
    u32x4 w[2][64];
    uint8_t sc[2][64];
    u32x4 x[UP ? 1 : 2][NT][256];
};

// Pieces are kept at the place of their index with some of its bits flipped
// by the row's, so that the 16 lanes that read one piece of 16 rows each meet
// different banks.
MOE_DEV int w4_wslot(int row, int blk) { return 4 * row + (blk ^ (row >> 2)); }
MOE_DEV int w4_xslot(int row, int piece) { return 16 * row + (piece ^ (4 * (row & 3) + (row >> 2))); }

// The lanes of a wave see each other's LDS writes in program order; this
// keeps the compiler to that order.
MOE_DEV void w4_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Steps [s, s + U) of a wave's reduction: all global loads, then step by step
// through LDS to the matrix units. Memory is read by quads of lanes, 64
// contiguous bytes of a row each: lane l takes row l / 4 of the weights and of
// the tokens, while the product wants row l % 16 (a load in the product's own
// order has a lane per row and costs the first-level cache four times the
// accesses). TAIL: blocks past the row's end count as zeros, of both operands.
template <bool UP, int NT, int U, bool TAIL>
MOE_DEV void w4_steps(int s, int nblk, const uint8_t *q0, const uint8_t *q1, const uint8_t *s0,
                      const uint8_t *s1, const uint16_t *const (&x)[2][NT], W4Stage<UP, NT> &st,
                      f32x4 (&acc)[2][NT]) {
    constexpr int P = UP ? 1 : 2;                 // h comes as two halves
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15, lr = lane >> 2, lc = lane & 3;
    u32x4 w[U][2], xr[U][P][NT][4];
    uint8_t sc[U][2];
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = 4 * (s + u) + lc;
        const bool ok = !TAIL || c < nblk;
        w[u][0] = w[u][1] = zero;
        sc[u][0] = sc[u][1] = 127;
        if (ok) {
            w[u][0] = *reinterpret_cast<const u32x4 *>(q0 + 16 * c);
            w[u][1] = *reinterpret_cast<const u32x4 *>(q1 + 16 * c);
            sc[u][0] = s0[c];
            sc[u][1] = s1[c];
        }
    }
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int p = 0; p < P; p++)
            if (x[p][t]) {
#pragma unroll
                for (int u = 0; u < U; u++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int c = 4 * (s + u) + j;
                        xr[u][p][t][j] = !TAIL || c < nblk
                            ? *reinterpret_cast<const u32x4 *>(x[p][t] + 32 * c + 8 * lc) : zero;
                    }
            }
#pragma unroll
    for (int u = 0; u < U; u++) {
        w4_lds_order();                           // the step before has been read
#pragma unroll
        for (int z = 0; z < 2; z++) {
            st.w[z][w4_wslot(lr, lc)] = w[u][z];
            st.sc[z][lane] = sc[u][z];
        }
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int p = 0; p < P; p++)
                if (x[p][t])
#pragma unroll
                    for (int j = 0; j < 4; j++) st.x[p][t][w4_xslot(lr, 4 * j + lc)] = xr[u][p][t][j];
        w4_lds_order();
        u32x4 a[2];
        float f[2];
#pragma unroll
        for (int z = 0; z < 2; z++) {
            a[z] = st.w[z][w4_wslot(i, g)];
            f[z] = __uint_as_float((uint32_t)st.sc[z][4 * i + g] << 23);
        }
#pragma unroll
        for (int m = 0; m < 4; m++) {
            const bf16x8 a0 = w4_widen(a[0][m], f[0]), a1 = w4_widen(a[1][m], f[1]);
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int p = 0; p < P; p++) {
                    const bf16x8 b = __builtin_bit_cast(bf16x8, st.x[p][t][w4_xslot(i, 4 * g + m)]);
                    acc[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, b, acc[0][t], 0, 0, 0);
                    acc[1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, b, acc[1][t], 0, 0, 0);
                }
        }
    }
}

// LDS of a workgroup: the waves' stages, then (SPLIT) their sums.
template <bool UP, int NT>
union W4Lds {
    W4Stage<UP, NT> stage[4];
    float red[4][2][256];
};

// N results of row `row`, columns from n: h as its two halves, or y.
template <bool UP, int N>
MOE_DEV void w4_store(const W4Args &p, int64_t row, int n, const float *v0, const float *v1) {
    if constexpr (UP) {
        uint16_t hi[N], lo[N];
#pragma unroll
        for (int q = 0; q < N; q++) {
            const float a = v0[q], e = expf(-0.5f * fabsf(a));
            const float o = (a < 0.f ? (a * e) * e : a) / fmaf(e, e, 1.f) * v1[q];
            hi[q] = f32_to_bf16(o);
            lo[q] = f32_to_bf16(o - bf16_to_f32(hi[q]));
        }
        __builtin_memcpy(p.hi_out + row * p.h + n, hi, sizeof(hi));
        __builtin_memcpy(p.lo_out + row * p.h + n, lo, sizeof(lo));
    } else {
        __builtin_memcpy(p.y + row * p.d + n, v0, N * sizeof(float));
        __builtin_memcpy(p.y + row * p.d + n + 16, v1, N * sizeof(float));
    }
}

// Rows [r, r + 16 NT) of the expert's rows [.., r1), two tiles of 16 weight
// rows: gate and up of 16 columns, or 32 rows of W2. SPLIT: a workgroup's
// four waves take a quarter of the reduction each and join their sums in LDS;
// otherwise each has tiles of its own. The columns of the product past the
// expert's last row hold what LDS held (a token is a column: it reaches no
// other) and are not stored.
template <bool UP, int NT, int U, bool SPLIT>
MOE_DEV void w4_rows(const W4Args &p, int64_t wrow0, int64_t wrow1, int n0, int r, int r1,
                     W4Lds<UP, NT> &lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = lane >> 2;
    const int nblk = p.K / 32;
    const uint8_t *q0 = p.wq + (wrow0 + lr) * (p.K / 2), *q1 = p.wq + (wrow1 + lr) * (p.K / 2);
    const uint8_t *s0 = p.ws + (wrow0 + lr) * nblk, *s1 = p.ws + (wrow1 + lr) * nblk;
    const uint16_t *x[2][NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int row = r + 16 * t + lr;
        x[0][t] = x[1][t] = nullptr;
        if (row < r1) {
            const int64_t src = (UP ? p.sorted_token[row] : row) * (int64_t)p.K;
            x[0][t] = p.x + src;
            x[1][t] = UP ? nullptr : p.lo + src;
        }
    }
    f32x4 acc[2][NT];
#pragma unroll
    for (int z = 0; z < 2; z++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[z][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int steps = (nblk + 3) / 4, part = SPLIT ? (steps + 3) / 4 : steps;
    int s = SPLIT ? wave * part : 0;
    const int end = min(s + part, steps), whole = min(end, nblk / 4);
    W4Stage<UP, NT> &st = lds.stage[wave];
    for (; s + U <= whole; s += U)
        w4_steps<UP, NT, U, false>(s, nblk, q0, q1, s0, s1, x, st, acc);
    for (; s < end; s++) w4_steps<UP, NT, 1, true>(s, nblk, q0, q1, s0, s1, x, st, acc);
    // lane: token lane % 16, weight rows 4 (lane / 16) .. + 3
    const int i = lane & 15, n4 = 4 * (lane >> 4);
    if constexpr (!SPLIT) {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int row = r + 16 * t + i;
            const float v0[4] = {acc[0][t][0], acc[0][t][1], acc[0][t][2], acc[0][t][3]};
            const float v1[4] = {acc[1][t][0], acc[1][t][1], acc[1][t][2], acc[1][t][3]};
            if (row < r1) w4_store<UP, 4>(p, row, n0 + n4, v0, v1);
        }
        return;
    }
#pragma unroll
    for (int t = 0; t < NT; t++) {
        __syncthreads();                          // the stages, or the tile before, have been read
#pragma unroll
        for (int z = 0; z < 2; z++) *reinterpret_cast<f32x4 *>(&lds.red[wave][z][i * 16 + n4]) = acc[z][t];
        __syncthreads();
        const int tid = threadIdx.x, row = r + 16 * t + (tid >> 4), n = tid & 15;
        float v[2];
#pragma unroll
        for (int z = 0; z < 2; z++)
            v[z] = (lds.red[0][z][tid] + lds.red[1][z][tid]) + (lds.red[2][z][tid] + lds.red[3][z][tid]);
        if (row < r1) w4_store<UP, 1>(p, row, n0 + n, &v[0], &v[1]);
    }
    __syncthreads();                              // the sums have been read
}

// blockIdx.y: rank of an expert with rows; blockIdx.x: 16 columns of h (UP) or
// 32 of d, without SPLIT four times as many, a quarter for each wave
template <bool UP, int NT, int U, bool SPLIT>
__global__ __launch_bounds__(256, NT == 1 ? 3 : 2) void w4_product(
    W4Args p, const int32_t *__restrict__ offsets, int E) {
    __shared__ W4Lds<UP, NT> lds;
    int e, r0, r1;
    if (!w4_active(offsets, E, blockIdx.y, e, r0, r1)) return;      // the whole workgroup
    const int tile = SPLIT ? blockIdx.x : 4 * blockIdx.x + (threadIdx.x >> 6);
    const int n0 = tile * (UP ? 16 : 32);
    if (!SPLIT && n0 >= (UP ? p.h : p.d)) return;                   // this wave alone: no barriers
    const int64_t base = (int64_t)e * (UP ? 2 * p.h : p.d);
    const int64_t w0 = base + n0, w1 = w0 + (UP ? p.h : 16);
    for (int r = r0; r < r1; r += 16 * NT) w4_rows<UP, NT, U, SPLIT>(p, w0, w1, n0, r, r1, lds);
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

#define SPLIT_MAX 2048
static size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// workspace: h's upper halves, its lower halves [R, h] bf16, y [R, d] fp32
size_t w4_ws_bytes(int64_t R, int d, int h) {
    return 2 * round256((size_t)R * h * 2) + round256((size_t)R * d * 4);
}

moe_status w4_experts_launch(const moe_w4_desc *w, hipStream_t s) {
    const int64_t R = w->T * w->k;
    char *ws = reinterpret_cast<char *>(w->ws);
    const size_t half = round256((size_t)R * w->h * 2);
    uint16_t *hi = reinterpret_cast<uint16_t *>(ws), *lo = reinterpret_cast<uint16_t *>(ws + half);
    float *y = reinterpret_cast<float *>(ws + 2 * half);
    const unsigned ny = (unsigned)(R < w->E ? R : w->E);
    const bool few = R <= 8 * (int64_t)w->E;
    const W4Args up = {reinterpret_cast<const uint16_t *>(w->x), nullptr, w->sorted_token, w->w1q,
                       w->w1_scale, hi, lo, nullptr, w->d, w->h, w->d};
    const W4Args down = {hi, lo, nullptr, w->w2q, w->w2_scale, nullptr, nullptr, y, w->h, w->h, w->d};
    const int nu = w->h / 16, nd = w->d / 32;
    if (!few)
        w4_product<true, 2, 2, false><<<dim3((nu + 3) / 4, ny), 256, 0, s>>>(up, w->offsets, w->E);
    else if ((int64_t)nu * ny <= SPLIT_MAX)
        w4_product<true, 1, 2, true><<<dim3(nu, ny), 256, 0, s>>>(up, w->offsets, w->E);
    else
        w4_product<true, 1, 2, false><<<dim3((nu + 3) / 4, ny), 256, 0, s>>>(up, w->offsets, w->E);
    if (!few)
        w4_product<false, 2, 1, false><<<dim3((nd + 3) / 4, ny), 256, 0, s>>>(down, w->offsets, w->E);
    else if ((int64_t)nd * ny <= SPLIT_MAX)
        w4_product<false, 1, 2, true><<<dim3(nd, ny), 256, 0, s>>>(down, w->offsets, w->E);
    else
        w4_product<false, 1, 2, false><<<dim3((nd + 3) / 4, ny), 256, 0, s>>>(down, w->offsets, w->E);
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
