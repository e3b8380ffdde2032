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

constexpr int kW4Unroll = 4;

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

// Steps [s, s + U) of a wave's reduction, blocks 4 s' + g of every row: all
// loads, then the products. TAIL: blocks past the row's end count as zeros
// (both operands, whatever x holds).
template <bool UP, int NT, int U, bool TAIL>
MOE_DEV void w4_steps(int s, int g, int nblk, const uint8_t *q0, const uint8_t *q1,
                      const uint8_t *s0, const uint8_t *s1, const uint16_t *const (&x)[NT],
                      const uint16_t *const (&xl)[NT], f32x4 (&acc)[2][NT]) {
    u32x4 w[U][2];
    uint32_t sc[U][2];
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int c = TAIL ? min(4 * (s + u) + g, nblk - 1) : 4 * (s + u) + g;
        w[u][0] = *reinterpret_cast<const u32x4 *>(q0 + 16 * c);
        w[u][1] = *reinterpret_cast<const u32x4 *>(q1 + 16 * c);
        sc[u][0] = s0[c];
        sc[u][1] = s1[c];
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        const bool ok = !TAIL || 4 * (s + u) + g < nblk;
        const int c = TAIL ? min(4 * (s + u) + g, nblk - 1) : 4 * (s + u) + g;
        const float f0 = __uint_as_float(sc[u][0] << 23), f1 = __uint_as_float(sc[u][1] << 23);
        const u32x4 w0 = ok ? w[u][0] : zero, w1 = ok ? w[u][1] : zero;
#pragma unroll
        for (int m = 0; m < 4; m++) {
            const bf16x8 a0 = w4_widen(w0[m], f0), a1 = w4_widen(w1[m], f1);
#pragma unroll
            for (int t = 0; t < NT; t++) {
                u32x4 v = *reinterpret_cast<const u32x4 *>(x[t] + 32 * c + 8 * m);
                v = ok ? v : zero;
                const bf16x8 b = __builtin_bit_cast(bf16x8, v);
                acc[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, b, acc[0][t], 0, 0, 0);
                acc[1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, b, acc[1][t], 0, 0, 0);
                if constexpr (!UP) {
                    u32x4 vl = *reinterpret_cast<const u32x4 *>(xl[t] + 32 * c + 8 * m);
                    vl = ok ? vl : zero;
                    const bf16x8 bl = __builtin_bit_cast(bf16x8, vl);
                    acc[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, bl, acc[0][t], 0, 0, 0);
                    acc[1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, bl, acc[1][t], 0, 0, 0);
                }
            }
        }
    }
}

// Rows [r, r + 16 NT) of the expert's rows [.., r1): two tiles of 16 weight
// rows (gate and up, or 32 rows of W2), the reduction in four parts, one a
// wave, joined in LDS. Lanes past the expert's last row compute the first
// row once more (a token is a column of the product: it reaches no other)
// and store nothing.
template <bool UP, int NT>
MOE_DEV void w4_rows(const W4Args &p, int64_t wrow0, int64_t wrow1, int n0, int r, int r1,
                     float (*red)[2][256]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i = lane & 15;
    const int nblk = p.K / 32;
    const uint8_t *q0 = p.wq + (wrow0 + i) * (p.K / 2), *q1 = p.wq + (wrow1 + i) * (p.K / 2);
    const uint8_t *s0 = p.ws + (wrow0 + i) * nblk, *s1 = p.ws + (wrow1 + i) * nblk;
    const uint16_t *x[NT], *xl[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int row = r + 16 * t + i < r1 ? r + 16 * t + i : r;
        const int64_t src = UP ? p.sorted_token[row] : row;
        x[t] = p.x + src * p.K;
        xl[t] = UP ? nullptr : p.lo + src * p.K;
    }
    f32x4 acc[2][NT];
#pragma unroll
    for (int z = 0; z < 2; z++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[z][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int steps = (nblk + 3) / 4, part = (steps + 3) / 4;
    int s = wave * part;
    const int end = min(s + part, steps), whole = min(end, nblk / 4);
    for (; s + kW4Unroll <= whole; s += kW4Unroll)
        w4_steps<UP, NT, kW4Unroll, false>(s, g, nblk, q0, q1, s0, s1, x, xl, acc);
    for (; s < end; s++) w4_steps<UP, NT, 1, true>(s, g, nblk, q0, q1, s0, s1, x, xl, acc);
    // lane: token i, weight rows 4 g .. 4 g + 3
#pragma unroll
    for (int t = 0; t < NT; t++) {
        __syncthreads();                          // the tile before has been read
#pragma unroll
        for (int z = 0; z < 2; z++)
            *reinterpret_cast<f32x4 *>(&red[wave][z][i * 16 + 4 * g]) = acc[z][t];
        __syncthreads();
        const int tid = threadIdx.x, row = r + 16 * t + (tid >> 4), n = tid & 15;
        float v[2];
#pragma unroll
        for (int z = 0; z < 2; z++)
            v[z] = (red[0][z][tid] + red[1][z][tid]) + (red[2][z][tid] + red[3][z][tid]);
        if (row >= r1) continue;
        if constexpr (UP) {
            const float a = v[0], e = expf(-0.5f * fabsf(a));
            const float o = (a < 0.f ? (a * e) * e : a) / fmaf(e, e, 1.f) * v[1];
            const uint16_t hi = f32_to_bf16(o);
            p.hi_out[(int64_t)row * p.h + n0 + n] = hi;
            p.lo_out[(int64_t)row * p.h + n0 + n] = f32_to_bf16(o - bf16_to_f32(hi));
        } else {
            p.y[(int64_t)row * p.d + n0 + n] = v[0];
            p.y[(int64_t)row * p.d + n0 + 16 + n] = v[1];
        }
    }
}

// blockIdx.x: 16 columns of h (UP) or 32 of d; blockIdx.y: rank of an expert with rows
template <bool UP>
__global__ __launch_bounds__(256) void w4_product(W4Args p, const int32_t *__restrict__ offsets,
                                                  int E) {
    __shared__ float red[4][2][256];
    int e, r0, r1;
    if (!w4_active(offsets, E, blockIdx.y, e, r0, r1)) return;      // the whole workgroup
    const int n0 = blockIdx.x * (UP ? 16 : 32);
    const int64_t base = (int64_t)e * (UP ? 2 * p.h : p.d);
    const int64_t w0 = base + n0, w1 = w0 + (UP ? p.h : 16);
    int r = r0;
    for (; r1 - r > 32; r += 64) w4_rows<UP, 4>(p, w0, w1, n0, r, r1, red);
    if (r1 - r > 16) w4_rows<UP, 2>(p, w0, w1, n0, r, r1, red);
    else if (r1 > r) w4_rows<UP, 1>(p, w0, w1, n0, r, r1, red);
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

moe_status w4_experts_launch(const moe_w4_desc *w, hipStream_t s) {
    const int64_t R = w->T * w->k;
    char *ws = reinterpret_cast<char *>(w->ws);
    const size_t half = round256((size_t)R * w->h * 2);
    uint16_t *hi = reinterpret_cast<uint16_t *>(ws), *lo = reinterpret_cast<uint16_t *>(ws + half);
    float *y = reinterpret_cast<float *>(ws + 2 * half);
    const unsigned ny = (unsigned)(R < w->E ? R : w->E);
    W4Args up = {reinterpret_cast<const uint16_t *>(w->x), nullptr, w->sorted_token, w->w1q, w->w1_scale,
                 hi, lo, nullptr, w->d, w->h, w->d};
    w4_product<true><<<dim3(w->h / 16, ny), 256, 0, s>>>(up, w->offsets, w->E);
    W4Args down = {hi, lo, nullptr, w->w2q, w->w2_scale, nullptr, nullptr, y, w->h, w->h, w->d};
    w4_product<false><<<dim3(w->d / 32, ny), 256, 0, s>>>(down, w->offsets, w->E);
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
