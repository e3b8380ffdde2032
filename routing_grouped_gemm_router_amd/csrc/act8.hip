// act8.hip -- 8-bit activation checkpoints (MXINT8, act8.h) and their use in
// the layer's backward pass.
//
// The layer's activations between forward and backward are what limits the
// batch (kongchang.com, "where the costs are": recomputing them saves about
// two thirds of that memory for about a fifth of the throughput). Kept in 8
// bits they take 33/64 of their bf16 size and nothing is computed twice but
// H' = silu(a) b, which follows from A||B. At T = 16384, d = 2048, h = 1024, E =
// 128, k = 4 in bf16 a layer holds 265 MiB instead of 897 and its forward plus
// backward takes 3.91 ms instead of 3.69 (recomputing holds 257 MiB and takes
// 4.40 ms).
//
// All kernels are bound by memory: each reads its inputs once and writes its
// outputs once, at a large copy's rate (4.7 to 5.2 TB/s here) or above it.
// What is read or written once and not soon again goes past the last-level
// cache (load_once, store_once): store 77 -> 68 us for 65536 rows of 2048 bf16
// (407 MB, 6.0 TB/s), combine with its checkpoint 125 -> 95 us. dy_perm is
// stored in the ordinary way: the GEMM that reads it comes next, and a layer's
// step gains nothing by the other (3.85 ms both ways), though combine and
// backward in turn would take 171 us instead of 177.
#include "act8.h"

namespace moe {

// vectors of each of a token's k rows in flight per thread (T = 16384, d = 2048,
// k = 4: combine 1 91 us, 2 95 us; backward 1 and 2 80 us, 4 83 us; T = 512, d =
// 4096, k = 8 backward 1 14.1 us, 2 12.3)
constexpr int kCombineU = 1, kCombineBwdU = 2;

// store: q, scale = checkpoint of in, a vector a thread (65536 x 2048 bf16: 68 us).
// Blocks of 32 lie in rows of a multiple
// of 32, so the matrix is one run of blocks.
template <bool BF16>
__global__ __launch_bounds__(256) void act8_store_vecs(const uint4 *__restrict__ in, int64_t n_vec,
                                                       typename Codes<BF16>::type *__restrict__ q,
                                                       uint8_t *__restrict__ scale) {
    typedef Row16<BF16> R;
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n_vec) return;                       // whole blocks of 32: n_vec % LPB == 0
    const uint4 w = load_once(in + v);
    const uint32_t sb = act8_scale_byte<BF16>(w);
    float f[R::N];
    R::unpack(w, f);
    typename Codes<BF16>::type c;
    act8_encode(f, sb, c);
    store_once(q + v, c);
    if (v % R::LPB == 0) scale[v / R::LPB] = (uint8_t)sb;
}

// load: the values a checkpoint stands for (65536 x 2048 bf16: 62 to 77 us)
template <bool BF16>
__global__ __launch_bounds__(256) void act8_load_vecs(const typename Codes<BF16>::type *__restrict__ q,
                                                      const uint8_t *__restrict__ scale,
                                                      int64_t n_vec, uint4 *__restrict__ out) {
    typedef Row16<BF16> R;
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n_vec) return;
    float f[R::N];
    act8_decode(q[v], act8_step(scale[v / R::LPB]), f);
    out[v] = R::pack(f);
}

// A||B and H' = silu(a) b from the checkpoint of A||B [rows, 2h]; hv = vectors
// of h. 65536 x 2048 bf16: 541 MB in 91 us, 5.9 TB/s.
template <bool BF16>
__global__ __launch_bounds__(256) void act8_swiglu_vecs(const typename Codes<BF16>::type *__restrict__ q,
                                                        const uint8_t *__restrict__ scale,
                                                        int64_t n_vec, int hv,
                                                        uint4 *__restrict__ ab,
                                                        uint4 *__restrict__ hp) {
    typedef Row16<BF16> R;
    const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (v >= n_vec) return;
    const int64_t row = v / hv;
    const int64_t va = v + row * hv, vb = va + hv;      // row * 2 hv + column
    float a[R::N], b[R::N], y[R::N];
    act8_decode(load_once(q + va), act8_step(scale[va / R::LPB]), a);
    act8_decode(load_once(q + vb), act8_step(scale[vb / R::LPB]), b);
    store_once(ab + va, R::pack(a));
    store_once(ab + vb, R::pack(b));
#pragma unroll
    for (int i = 0; i < R::N; i++) y[i] = silu(a[i]) * b[i];
    store_once(hp + v, R::pack(y));
}

// The combine kernels give a token G threads: less than a wave for narrow
// rows, whole workgroups for wide rows of few tokens.
template <int G>
MOE_DEV int64_t token_of_group() {
    return G >= 256 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
}

// Each of N values summed over the G threads of a token, in a fixed order; all
// of them get the sums.
template <int G, int N>
MOE_DEV void group_sums(float (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N; j++) {
        if constexpr (G >= 64) v[j] = wave_sum(v[j]);
        else
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) v[j] += __shfl_xor(v[j], o);
    }
    if constexpr (G > 64) {
        __shared__ float part[G / 64][N];
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int j = 0; j < N; j++) part[threadIdx.x / 64][j] = v[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; j++) {
            v[j] = part[0][j];
            for (int w = 1; w < G / 64; w++) v[j] += part[w][j];
        }
    }
}

// combine that keeps the experts' rows: out[t] = sum_j g[t,j] y[token_pos[t,j]]
// (fp32 sum, ascending j) and the checkpoint of every row it reads, from one
// read: 474 MB at T = 16384, d = 2048, k = 4 bf16 in 95 us after its
// backward's dirty lines, 80 without (5.0 to 5.9 TB/s), where the combine alone takes 61 and
// a store of its own 68.
template <bool BF16, int KMAX, int U, int G>
__global__ __launch_bounds__(G > 256 ? G : 256) void combine_act8_rows(
    const uint4 *__restrict__ y, const float *__restrict__ gate,
    const int32_t *__restrict__ token_pos, int64_t T, int nv, int k, uint4 *__restrict__ out,
    typename Codes<BF16>::type *__restrict__ y8, uint8_t *__restrict__ y8_scale) {
    typedef Row16<BF16> R;
    const int lane = threadIdx.x % G;
    const int64_t t = token_of_group<G>();
    if (t >= T) return;
    int32_t pos[KMAX];
    float g[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; j++) {
        pos[j] = j < k ? token_pos[t * k + j] : -1;
        g[j] = j < k ? gate[t * k + j] : 0.f;
    }
    for (int c0 = lane; c0 < nv; c0 += G * U) {
        uint4 w[U][KMAX];
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int j = 0; j < KMAX; j++)
                if (c0 + G * u < nv && pos[j] >= 0) w[u][j] = load_once(y + (int64_t)pos[j] * nv + c0 + G * u);
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = c0 + G * u;
            if (c >= nv) break;
            float acc[R::N];
#pragma unroll
            for (int i = 0; i < R::N; i++) acc[i] = 0.f;
#pragma unroll
            for (int j = 0; j < KMAX; j++) {
                if (pos[j] < 0) continue;                   // dropped row
                const int64_t v = (int64_t)pos[j] * nv + c;
                const uint32_t sb = act8_scale_byte<BF16>(w[u][j]);
                float f[R::N];
                R::unpack(w[u][j], f);
                typename Codes<BF16>::type q;
                act8_encode(f, sb, q);
                store_once(y8 + v, q);
                if (c % R::LPB == 0) y8_scale[v / R::LPB] = (uint8_t)sb;
#pragma unroll
                for (int i = 0; i < R::N; i++) acc[i] = fmaf(g[j], f[i], acc[i]);
            }
            out[t * nv + c] = R::pack(acc);
        }
    }
}

// combine backward with the router backward, the experts' rows read from
// their checkpoint:
//   dg_j = <dOut[t], y8[p_j]>,  dy_perm[p_j] = round(g_j dOut[t]),
//   dlogits[t, e_j] = g_j sum_i g_i (dg_j - dg_i), 0 for unselected experts
// (the gates sum to one; this form has no cancellation between large terms).
// ROWS = false (the MXFP8 backward, whose quantiser forms dy_perm itself):
// row_gate[p_j] = g_j instead of dy_perm's rows. 484 MB at T = 16384, d = 2048, k
// = 4 bf16 in 93 us after the forward (81 to 98; 5.2 TB/s); from bf16 rows it takes 100.
template <bool BF16, int KMAX, int U, bool ROWS, int G>
__global__ __launch_bounds__(G > 256 ? G : 256) void combine_bwd_act8_rows(
    const uint4 *__restrict__ dout, const typename Codes<BF16>::type *__restrict__ y8,
    const uint8_t *__restrict__ y8_scale, const float *__restrict__ gate,
    const int32_t *__restrict__ topk_idx, const int32_t *__restrict__ token_pos, int64_t T, int nv,
    int k, int E, uint4 *__restrict__ dy, float *__restrict__ row_gate,
    float *__restrict__ dlogits, float *__restrict__ dgate) {
    typedef Row16<BF16> R;
    const int lane = threadIdx.x % G;
    const int64_t t = token_of_group<G>();
    if (t >= T) return;                           // whole groups
    int32_t pos[KMAX], ex[KMAX];
    float g[KMAX], dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; j++) {
        pos[j] = j < k ? token_pos[t * k + j] : -1;
        ex[j] = j < k ? topk_idx[t * k + j] : -1;
        g[j] = j < k ? gate[t * k + j] : 0.f;
        dot[j] = 0.f;
    }
    for (int c0 = lane; c0 < nv; c0 += G * U) {
        uint4 wo[U];
        typename Codes<BF16>::type q[U][KMAX];
        uint8_t sc[U][KMAX];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = c0 + G * u;
            if (c >= nv) break;
            wo[u] = load_once(dout + t * nv + c);
#pragma unroll
            for (int j = 0; j < KMAX; j++) {
                if (pos[j] < 0) continue;
                const int64_t v = (int64_t)pos[j] * nv + c;
                q[u][j] = load_once(y8 + v);
                sc[u][j] = y8_scale[v / R::LPB];
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = c0 + G * u;
            if (c >= nv) break;
            float fo[R::N];
            R::unpack(wo[u], fo);
#pragma unroll
            for (int j = 0; j < KMAX; j++) {
                if (pos[j] < 0) continue;
                float fy[R::N], fd[R::N];
                act8_decode(q[u][j], act8_step(sc[u][j]), fy);
#pragma unroll
                for (int i = 0; i < R::N; i++) {
                    dot[j] = fmaf(fo[i], fy[i], dot[j]);
                    fd[i] = g[j] * fo[i];
                }
                if constexpr (ROWS) dy[(int64_t)pos[j] * nv + c] = R::pack(fd);
            }
        }
    }
    group_sums<G>(dot);
#pragma unroll
    for (int j = 0; j < KMAX; j++)
        if (pos[j] < 0) dot[j] = 0.f;   // dropped row: its gate had no effect
    float rg[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; j++) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < KMAX; i++) s = fmaf(g[i], dot[j] - dot[i], s);
        rg[j] = g[j] * s;
    }
    for (int e = lane; e < E; e += G) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < KMAX; j++)
            if (ex[j] == e) v = rg[j];
        dlogits[t * E + e] = v;
    }
    if (lane == 0) {
#pragma unroll
        for (int j = 0; j < KMAX; j++) {
            if (dgate && j < k) dgate[t * k + j] = dot[j];
            if (!ROWS && pos[j] >= 0) row_gate[pos[j]] = g[j];
        }
    }
}

// ---------------------------------------------------------------------------
// launchers

moe_status act8_store_launch(const void *in, moe_dtype dt, int64_t rows, int64_t cols, uint8_t *q,
                             uint8_t *scale, hipStream_t s) {
    const bool bf = dt == MOE_BF16;
    const int64_t n_vec = rows * (cols / (bf ? 8 : 4));
    for (int64_t at = 0; at < n_vec; at += kMaxBlocks * 256) {
        const int64_t n = n_vec - at < kMaxBlocks * 256 ? n_vec - at : kMaxBlocks * 256;
        const unsigned nb = (unsigned)((n + 255) / 256);
        const uint4 *src = reinterpret_cast<const uint4 *>(in) + at;
        if (bf)
            act8_store_vecs<true><<<nb, 256, 0, s>>>(src, n, reinterpret_cast<uint2 *>(q) + at,
                                                     scale + at / 4);
        else
            act8_store_vecs<false><<<nb, 256, 0, s>>>(src, n, reinterpret_cast<uint32_t *>(q) + at,
                                                      scale + at / 8);
    }
    return launch_status();
}

moe_status act8_load_launch(const uint8_t *q, const uint8_t *scale, moe_dtype dt, int64_t rows,
                            int64_t cols, void *out, hipStream_t s) {
    const bool bf = dt == MOE_BF16;
    const int64_t n_vec = rows * (cols / (bf ? 8 : 4));
    for (int64_t at = 0; at < n_vec; at += kMaxBlocks * 256) {
        const int64_t n = n_vec - at < kMaxBlocks * 256 ? n_vec - at : kMaxBlocks * 256;
        const unsigned nb = (unsigned)((n + 255) / 256);
        uint4 *dst = reinterpret_cast<uint4 *>(out) + at;
        if (bf)
            act8_load_vecs<true><<<nb, 256, 0, s>>>(reinterpret_cast<const uint2 *>(q) + at,
                                                    scale + at / 4, n, dst);
        else
            act8_load_vecs<false><<<nb, 256, 0, s>>>(reinterpret_cast<const uint32_t *>(q) + at,
                                                     scale + at / 8, n, dst);
    }
    return launch_status();
}

moe_status act8_swiglu_launch(const uint8_t *q, const uint8_t *scale, moe_dtype dt, int64_t rows,
                              int h, void *ab, void *hp, hipStream_t s) {
    const bool bf = dt == MOE_BF16;
    const int hv = h / (bf ? 8 : 4);
    const int64_t step = kMaxBlocks * 256 / hv;        // rows of a launch
    for (int64_t r = 0; r < rows; r += step) {
        const int64_t n = (rows - r < step ? rows - r : step) * hv;
        const unsigned nb = (unsigned)((n + 255) / 256);
        uint4 *a = reinterpret_cast<uint4 *>(ab) + r * 2 * hv, *y = reinterpret_cast<uint4 *>(hp) + r * hv;
        const uint8_t *qq = q + r * 2 * h, *ss = scale + r * 2 * h / 32;
        if (bf)
            act8_swiglu_vecs<true><<<nb, 256, 0, s>>>(reinterpret_cast<const uint2 *>(qq), ss, n, hv, a, y);
        else
            act8_swiglu_vecs<false><<<nb, 256, 0, s>>>(reinterpret_cast<const uint32_t *>(qq), ss, n, hv, a, y);
    }
    return launch_status();
}

// Threads of a token, nv vectors of 16 bytes a row (bf16, T = 32768, k = 8 unless
// said):
//  - 16 for rows of up to 16 vectors (d = 64: forward 21 us against 58 with a
//    wave, backward 27 against 70), and up to 32 where the tokens fill the chip (d
//    = 256: 47 against 71, 45 against 75; T = 4096, k = 4: 5.8 against 5.2);
//  - forward: a workgroup of 256 from 128 vectors (d = 2048: 306 against 354; T =
//    512: 7.4 against 17; d = 512: 97 against 86), of 1024 from 1024 (d = 8192: 1407
//    against 1498; T = 512: 24 against 31; d = 2048: 445 against 360);
//  - backward, whose sums cross the waves: a workgroup of 256 from 256 vectors if
//    each thread has four or more (d = 4096: 706 against 748; d = 2048, k = 1: 60
//    against 55; at the border, T = 16384, d = 2048, k = 4: 94.5 against 102, with
//    its forward 189 against 197; fp32 d = 1024: 83 against 93; below it, k = 2:
//    56 against 59, and d = 1024, k = 8: 118 against 95), or from 128 where the
//    waves of the tokens alone do not fill the chip (T = 512, d = 2048: 8.3 against
//    10.9; d = 16384: 40 against 63).
static int combine_group(int nv, int64_t T, int k, bool backward) {
    if (nv <= 16 || (nv <= 32 && T >= 16384)) return 16;
    if (!backward) return nv >= 1024 ? 1024 : nv >= 128 ? 256 : 64;
    return (nv >= 256 && nv * k >= 1024) || (nv >= 128 && T <= 2048) ? 256 : 64;
}

#define ACT8_KSWITCH(G, k, F) \
    ((k) <= 1 ? F(1, G) : (k) <= 2 ? F(2, G) : (k) <= 4 ? F(4, G) : F(8, G))

template <bool BF16>
static void combine_act8_run(const void *y, const float *gate, const int32_t *token_pos, int64_t T,
                             int d, int k, void *out, uint8_t *y8, uint8_t *y8_scale,
                             hipStream_t s) {
    typedef typename Codes<BF16>::type C;
    const int nv = d / Row16<BF16>::N, group = combine_group(nv, T, k, false);
    const int tokens = group < 256 ? 256 / group : 1, threads = group < 256 ? 256 : group;
    for (int64_t t = 0; t < T; t += kMaxBlocks * tokens) {
        const int64_t n = T - t < kMaxBlocks * tokens ? T - t : kMaxBlocks * tokens;
        const unsigned nb = (unsigned)((n + tokens - 1) / tokens);
#define L(K, G)                                                                                  \
    (combine_act8_rows<BF16, K, kCombineU, G><<<nb, threads, 0, s>>>(                            \
         reinterpret_cast<const uint4 *>(y), gate + t * k, token_pos + t * k, n, nv, k,          \
         reinterpret_cast<uint4 *>(out) + t * nv, reinterpret_cast<C *>(y8), y8_scale), 0)
        group == 16 ? ACT8_KSWITCH(16, k, L) : group == 64 ? ACT8_KSWITCH(64, k, L)
            : group == 256 ? ACT8_KSWITCH(256, k, L) : ACT8_KSWITCH(1024, k, L);
#undef L
    }
}

moe_status combine_act8_launch(const void *y, moe_dtype dt, const float *gate,
                               const int32_t *token_pos, int64_t T, int d, int k, void *out,
                               uint8_t *y8, uint8_t *y8_scale, hipStream_t s) {
    if (dt == MOE_BF16) combine_act8_run<true>(y, gate, token_pos, T, d, k, out, y8, y8_scale, s);
    else combine_act8_run<false>(y, gate, token_pos, T, d, k, out, y8, y8_scale, s);
    return launch_status();
}

template <bool BF16, bool ROWS>
static void combine_bwd_act8_run(const void *dout, const uint8_t *y8, const uint8_t *y8_scale,
                                 const float *gate, const int32_t *topk_idx,
                                 const int32_t *token_pos, int64_t T, int d, int k, int E, void *dy,
                                 float *row_gate, float *dlogits, float *dgate, hipStream_t s) {
    typedef typename Codes<BF16>::type C;
    const int nv = d / Row16<BF16>::N, group = combine_group(nv, T, k, true);
    const int tokens = group < 256 ? 256 / group : 1, threads = group < 256 ? 256 : group;
    for (int64_t t = 0; t < T; t += kMaxBlocks * tokens) {
        const int64_t n = T - t < kMaxBlocks * tokens ? T - t : kMaxBlocks * tokens;
        const unsigned nb = (unsigned)((n + tokens - 1) / tokens);
#define L(K, G)                                                                                   \
    (combine_bwd_act8_rows<BF16, K, kCombineBwdU, ROWS, G><<<nb, threads, 0, s>>>(                \
         reinterpret_cast<const uint4 *>(dout) + t * nv, reinterpret_cast<const C *>(y8),         \
         y8_scale, gate + t * k, topk_idx + t * k, token_pos + t * k, n, nv, k, E,                \
         reinterpret_cast<uint4 *>(dy), row_gate, dlogits + t * E, dgate ? dgate + t * k : nullptr), 0)
        group == 16 ? ACT8_KSWITCH(16, k, L) : group == 64 ? ACT8_KSWITCH(64, k, L)
            : ACT8_KSWITCH(256, k, L);
#undef L
    }
}

// dy: the rows of dy_perm; without it (bf16) row_gate: each routed row's gate.
moe_status combine_bwd_act8_launch(const void *dout, moe_dtype dt, const uint8_t *y8,
                                   const uint8_t *y8_scale, const float *gate,
                                   const int32_t *topk_idx, const int32_t *token_pos, int64_t T,
                                   int d, int k, int E, void *dy, float *row_gate, float *dlogits,
                                   float *dgate, hipStream_t s) {
    if (dt == MOE_F32)
        combine_bwd_act8_run<false, true>(dout, y8, y8_scale, gate, topk_idx, token_pos, T, d, k, E,
                                          dy, nullptr, dlogits, dgate, s);
    else if (dy)
        combine_bwd_act8_run<true, true>(dout, y8, y8_scale, gate, topk_idx, token_pos, T, d, k, E,
                                         dy, nullptr, dlogits, dgate, s);
    else
        combine_bwd_act8_run<true, false>(dout, y8, y8_scale, gate, topk_idx, token_pos, T, d, k, E,
                                          nullptr, row_gate, dlogits, dgate, s);
    return launch_status();
}

}  // namespace moe
