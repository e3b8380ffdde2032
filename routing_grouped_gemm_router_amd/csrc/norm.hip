// norm.hip -- layer norm and root-mean-square norm, forward and backward.
//
//   s = x (+ res),  mu = mean(s),  r = 1 / sqrt(mean((s - mu)^2) + eps)
//   y = (s - mu) r gamma + beta
// and, with g = dy gamma and xh = (s - mu) r,
//   dx = r (g - mean(g) - xh mean(g xh)) (+ dsum),
//   dgamma = sum_t dy xh,  dbeta = sum_t dy.
// The root-mean-square norm (RMS) is the same without a mean and without beta:
//   r = 1 / sqrt(mean(s^2) + eps),  y = s r gamma,
//   dx = r (g - xh mean(g xh)) (+ dsum),  dgamma = sum_t dy xh,  xh = s r.
// It can write y as MXFP8 too, or alone (mx_encode.h), the rows that the 8-bit
// experts take: the bytes that quantising the stored y gives.
// s may be kept between the two passes as an 8-bit checkpoint (act8.h),
// written from the forward's registers and read by the backward in place of
// s. All sums and statistics are fp32, in a fixed order (no atomics), but for
// the root-mean-square norm's forward, which joins its threads' fp32 sums and
// takes their root in fp64; the variance is taken about the mean, from the row in
// registers.
//
// Both passes are bound by memory and read and write every row once; a row
// stays in its threads' registers from its load to its last store, in its own
// type (unpacking a bf16 again is cheaper than holding it as fp32). The rate is
// a large copy's, 4.7 to 5.2 TB/s on this card: 16384 x 2048 bf16 with a
// residual and a checkpoint, forward 303 MB in 57 us (5.3 TB/s), backward from
// the checkpoint with a stream gradient 236 MB in 47 us (5.0 TB/s) and 4.5 us for
// the weights' sums; 32768 x 4096 201 and 185 us (6.0 and 5.1 TB/s); over widths
// from 32 to 16384, 256 MiB of rows: 4.4 to 5.4 TB/s forward, 3.4 to 4.9 backward
// (the ends of the backward's range: few columns a thread to sum over, or no
// registers to load ahead). The root-mean-square norm: 16384 x 2048 bf16 with a
// residual, into s, y and MXFP8 55 us (304 MB, 5.5 TB/s), backward with a stream
// gradient 46 us (5.9 TB/s) and 4 us for the weights' sum; 8192 x 4096 into s and
// MXFP8 alone 44 us (236 MB, 5.4 TB/s); one row of 2048 1.9 us.
#include <type_traits>

#include "act8.h"
#include "mx_encode.h"

namespace moe {

// The MXFP8 bytes and scale of this lane's vector of a block of 32 (f: its
// elements as the norm's type rounds them). The block's 4 (bf16) or 8 (fp32)
// neighbouring lanes must be active.
template <bool BF16>
MOE_DEV uint32_t mx_encode_vec(const float *f, typename Codes<BF16>::type &q) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < Row16<BF16>::N; e++) m = fmaxf(m, fabsf(f[e]));
    m = fmaxf(m, dpp_move<kDppXor1>(m));
    m = fmaxf(m, dpp_move<kDppXor2>(m));
    if constexpr (!BF16) m = fmaxf(m, dpp_move<kDppHalfMirror>(m));
    const uint32_t sb = mx_scale_byte(m);
    if constexpr (BF16) {
        q.x = e4m3x4(f[0], f[1], f[2], f[3], sb);
        q.y = e4m3x4(f[4], f[5], f[6], f[7], sb);
    } else
        q = e4m3x4(f[0], f[1], f[2], f[3], sb);
    return sb;
}

// Sum of v over the threads of a row within their wave: G = 4, 8, 16, 32 or
// all 64 neighbouring lanes (G >= 64).
MOE_DEV float swap16_sum(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
MOE_DEV float swap32_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
MOE_DEV double swap16_sum(double v) {
    const auto l = __builtin_amdgcn_permlane16_swap(__double2loint(v), __double2loint(v), false, false);
    const auto h = __builtin_amdgcn_permlane16_swap(__double2hiint(v), __double2hiint(v), false, false);
    return __hiloint2double(h[0], l[0]) + __hiloint2double(h[1], l[1]);
}
MOE_DEV double swap32_sum(double v) {
    const auto l = __builtin_amdgcn_permlane32_swap(__double2loint(v), __double2loint(v), false, false);
    const auto h = __builtin_amdgcn_permlane32_swap(__double2hiint(v), __double2hiint(v), false, false);
    return __hiloint2double(h[0], l[0]) + __hiloint2double(h[1], l[1]);
}
template <int CTRL>
MOE_DEV double dpp_move(double v) {
    return __hiloint2double(dpp_move<CTRL>(__double2hiint(v)), dpp_move<CTRL>(__double2loint(v)));
}
template <int G, typename F>
MOE_DEV F group_sum(F v) {
    v += dpp_move<kDppXor1>(v);
    v += dpp_move<kDppXor2>(v);
    if constexpr (G >= 8) v += dpp_move<kDppHalfMirror>(v);
    if constexpr (G >= 16) v += dpp_move<kDppRowRor8>(v);
    if constexpr (G >= 32) v = swap16_sum(v);
    if constexpr (G >= 64) v = swap32_sum(v);
    return v;
}

// The waves' sums of a row that is a workgroup (G = 256, 512 or 1024
// threads), added in a fixed order.
template <int G, typename F>
MOE_DEV F waves_sum(const F *q) {
    F v = 0;
#pragma unroll
    for (int i = 0; i < G / 64; i += 4) v += (q[i] + q[i + 1]) + (q[i + 2] + q[i + 3]);
    return v;
}

// Sum over the row's G threads (red: G / 64 values in LDS, its own for every
// call between two barriers of the row).
template <int G, typename F>
MOE_DEV F row_sum(F v, F *red) {
    v = group_sum<G>(v);
    if constexpr (G >= 256) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = waves_sum<G>(red);
    }
    return v;
}

// threads of a workgroup: its rows are G threads each
constexpr int norm_threads(int g) { return g > 256 ? g : 256; }

template <bool BF16>
MOE_DEV void load_params(const float *p, int c, float *f) {
    const float4 *q = reinterpret_cast<const float4 *>(p) + (int64_t)c * (Row16<BF16>::N / 4);
#pragma unroll
    for (int i = 0; i < Row16<BF16>::N / 4; i++) {
        const float4 v = q[i];
        f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
    }
}

// 1 / sqrt(a) in two parts whose sum is off by some 2^-45 of it: the hardware's
// reciprocal root and one step of Newton's iteration, whose residual 1 - a r^2 the
// fused products give exactly. Where a or r^2 leaves fp32's range, lo is 0.
MOE_DEV void rsqrt_hi_lo(double a, float &hi, float &lo) {
    const float ah = (float)a, al = (float)(a - (double)ah);
    // (the instruction takes subnormal numbers as zeros)
    const float r = ah < 1e-36f ? 1.f / sqrtf(ah) : __builtin_amdgcn_rsqf(ah), q = r * r;
    float e = fmaf(-ah, q, 1.f);
    e = fmaf(-ah, fmaf(r, r, -q), e);
    e = fmaf(-al, q, e);
    const float c = fabsf(e) < 1e-3f ? 0.5f * r * e : 0.f;
    hi = r + c;
    lo = c == 0.f ? 0.f : (r - hi) + c;
}

// G threads a row, V 16-byte vectors a thread (vector lane + i G of the row).
// RMS: no mean (and none stored), no beta; y may be null if yq is not. A row's sum
// is joined in fp64 and s r gamma rounded once, to fp32, in front of y's own
// rounding: an element of y on the wrong side of a bf16 step may be one of yq on
// the wrong side of an E4M3 step, a sixteenth of its value. What it takes more
// than two products an element hides behind the loads.
template <bool BF16, int G, int V, bool RMS>
__global__ __launch_bounds__(norm_threads(G)) void norm_fwd(
    const uint4 *__restrict__ x, const uint4 *__restrict__ res, const float *__restrict__ gamma,
    const float *__restrict__ beta, float eps, int64_t T, int nv,
    typename std::conditional<RMS, double, float>::type inv_d, uint4 *__restrict__ y,
    uint4 *__restrict__ sum, float *__restrict__ mean,
    float *__restrict__ rstd, typename Codes<BF16>::type *__restrict__ x8,
    uint8_t *__restrict__ x8_scale, typename Codes<BF16>::type *__restrict__ yq,
    uint8_t *__restrict__ yq_scale) {
    typedef Row16<BF16> R;
    typedef typename std::conditional<RMS, double, float>::type Sum;
    __shared__ Sum red[RMS ? 1 : 2][16];
    const int lane = threadIdx.x % G;
    const int64_t t = (int64_t)blockIdx.x * (norm_threads(G) / G) + threadIdx.x / G;
    if (t >= T) return;                         // G >= 256: never (one row a workgroup)
    const int64_t base = t * nv;
    uint4 w[V];
    float s1 = 0.f;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = lane + i * G;
        w[i] = make_uint4(0, 0, 0, 0);
        if (c >= nv) continue;
        w[i] = x[base + c];
        float f[R::N];
        R::unpack(w[i], f);
        if (res) {
            float q[R::N];
            R::unpack(res[base + c], q);
#pragma unroll
            for (int e = 0; e < R::N; e++) f[e] += q[e];
            w[i] = R::pack(f);                  // the stream in its own type: what the norm sees
            sum[base + c] = w[i];
            R::unpack(w[i], f);
        }
#pragma unroll
        for (int e = 0; e < R::N; e++) s1 = RMS ? fmaf(f[e], f[e], s1) : s1 + f[e];
    }
    float mu = 0.f, r, rl = 0.f;
    if constexpr (RMS) {
        rsqrt_hi_lo(fma(row_sum<G>((double)s1, red[0]), inv_d, (double)eps), r, rl);
    } else {
        s1 = row_sum<G>(s1, red[0]);
        mu = s1 * inv_d;
        float s2 = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            if (lane + i * G >= nv) continue;
            float f[R::N];
            R::unpack(w[i], f);
#pragma unroll
            for (int e = 0; e < R::N; e++) s2 = fmaf(f[e] - mu, f[e] - mu, s2);
        }
        s2 = row_sum<G>(s2, red[1]);
        r = 1.f / sqrtf(fmaf(s2, inv_d, eps));
    }
    if (lane == 0) {
        if (!RMS && mean) mean[t] = mu;
        if (rstd) rstd[t] = r;
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = lane + i * G;
        if (c >= nv) continue;
        float f[R::N], ga[R::N], o[R::N];
        R::unpack(w[i], f);
        load_params<BF16>(gamma, c, ga);
#pragma unroll
        for (int e = 0; e < R::N; e++) {
            if constexpr (RMS) {
                // (f r + l) gamma; l gamma held in range for the sake of an infinite gamma
                const float h = f[e] * r, l = fmaf(f[e], rl, fmaf(f[e], r, -h));
                o[e] = fmaf(h, ga[e], __builtin_amdgcn_fmed3f(l * ga[e], -3e38f, 3e38f));
            } else
                o[e] = (f[e] - mu) * r * ga[e];
        }
        if (!RMS && beta) {
            load_params<BF16>(beta, c, ga);
#pragma unroll
            for (int e = 0; e < R::N; e++) o[e] += ga[e];
        }
        const uint4 p = R::pack(o);
        if (!RMS || y) y[base + c] = p;
        if (RMS && yq) {
            typename Codes<BF16>::type q;
            R::unpack(p, o);
            const uint32_t sb = mx_encode_vec<BF16>(o, q);
            yq[base + c] = q;
            if (c % R::LPB == 0) yq_scale[(base + c) / R::LPB] = (uint8_t)sb;
        }
        if (x8) {
            const uint32_t sb = act8_scale_byte<BF16>(w[i]);
            typename Codes<BF16>::type q;
            act8_encode(f, sb, q);
            x8[base + c] = q;
            if (c % R::LPB == 0) x8_scale[(base + c) / R::LPB] = (uint8_t)sb;
        }
    }
}

// What a thread reads of one row in the backward pass.
template <bool BF16, int V, bool CKPT>
struct NormRow {
    typedef typename Codes<BF16>::type C;
    uint4 dy[V], ds[V], x[CKPT ? 1 : V];
    C q[CKPT ? V : 1];
    uint8_t sc[CKPT ? V : 1];
    float mu, r;
};

// Backward: every workgroup takes rows blockIdx.x * RPB + ..., strided by the
// grid, keeps its sums of dy xh and dy in registers and leaves them in
// part[blockIdx.x][0..1][d]. A row's loads are issued before the row in front
// of it is computed: with two workgroups a compute unit (so that the partial
// sums stay small) nothing else would hide the two reductions of a row (16384 x
// 2048 74.7 -> 53.4 us, 32768 x 4096 267 -> 180 us).
// RMS: mean is not read, and the workgroups leave part[blockIdx.x][d]. ONCE: the
// rows are read past the last-level cache (kOnceBytes).
template <bool BF16, int G, int V, bool CKPT, bool RMS, bool ONCE>
__global__ __launch_bounds__(norm_threads(G)) void norm_bwd(
    const uint4 *__restrict__ dy, const uint4 *__restrict__ x,
    const typename Codes<BF16>::type *__restrict__ x8, const uint8_t *__restrict__ x8_scale,
    const float *__restrict__ mean, const float *__restrict__ rstd,
    const float *__restrict__ gamma, const uint4 *__restrict__ dsum, int64_t T, int nv, float inv_d,
    uint4 *__restrict__ dx, float *__restrict__ part) {
    typedef Row16<BF16> R;
    constexpr int RPB = norm_threads(G) / G;
    __shared__ float red[2][2][16];
    __shared__ float acc_s[G >= 256 ? 1 : 256 * R::N];
    const int lane = threadIdx.x % G;
    // a workgroup of 1024 threads has 128 registers a thread: it does not load
    // ahead, and with 16 elements a thread it does not keep gamma either (d
    // fp32 that stay in the caches)
    constexpr bool LEAN = G == 1024, RELOAD = LEAN && V * R::N == 16;
    float dg[V * R::N], db[V * R::N], ga[V * R::N];
#pragma unroll
    for (int i = 0; i < V; i++) {
#pragma unroll
        for (int e = 0; e < R::N; e++) dg[i * R::N + e] = db[i * R::N + e] = 0.f;
        if (!RELOAD && lane + i * G < nv) load_params<BF16>(gamma, lane + i * G, ga + i * R::N);
    }
    typedef NormRow<BF16, V, CKPT> Row;
    auto load = [&](Row &w, int64_t t) {
        if (t >= T) return;
        const int64_t base = t * nv;
        w.mu = RMS ? 0.f : mean[t];
        w.r = rstd[t];
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = lane + i * G;
            if (c >= nv) continue;
            w.dy[i] = ONCE ? load_once(dy + base + c) : dy[base + c];
            if constexpr (CKPT) {
                w.q[i] = x8[base + c];
                w.sc[i] = x8_scale[(base + c) / R::LPB];
            } else
                w.x[i] = ONCE ? load_once(x + base + c) : x[base + c];
            if (dsum) w.ds[i] = ONCE ? load_once(dsum + base + c) : dsum[base + c];
        }
    };
    int par = 0;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / G;
    Row next;
    if (!LEAN) load(next, t);
    for (; t < T; t += step, par ^= 1) {
        if (LEAN) load(next, t);
        const Row w = next;
        if (!LEAN) load(next, t + step);
        const int64_t base = t * nv;
        float xh[V * R::N];
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            if (lane + i * G >= nv) continue;
            float f[R::N], g[R::N];
            if constexpr (CKPT) act8_decode(w.q[i], act8_step(w.sc[i]), f);
            else R::unpack(w.x[i], f);
            R::unpack(w.dy[i], g);
            if (RELOAD) load_params<BF16>(gamma, lane + i * G, ga + i * R::N);
#pragma unroll
            for (int e = 0; e < R::N; e++) {
                const float h = (RMS ? f[e] : f[e] - w.mu) * w.r;
                xh[i * R::N + e] = h;
                dg[i * R::N + e] = fmaf(g[e], h, dg[i * R::N + e]);
                const float gw = g[e] * ga[i * R::N + e];
                if constexpr (!RMS) {
                    db[i * R::N + e] += g[e];
                    c1 += gw;
                }
                c2 = fmaf(gw, h, c2);
            }
        }
        if constexpr (!RMS) c1 = group_sum<G>(c1);
        c2 = group_sum<G>(c2);
        if constexpr (G >= 256) {
            // one barrier a row: the next row writes the other half
            if ((threadIdx.x & 63) == 0) {
                if constexpr (!RMS) red[par][0][threadIdx.x >> 6] = c1;
                red[par][1][threadIdx.x >> 6] = c2;
            }
            __syncthreads();
            if constexpr (!RMS) c1 = waves_sum<G>(red[par][0]);
            c2 = waves_sum<G>(red[par][1]);
        }
        c1 *= inv_d;
        c2 *= inv_d;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = lane + i * G;
            if (c >= nv) continue;
            float g[R::N], o[R::N];
            R::unpack(w.dy[i], g);
            if (RELOAD) load_params<BF16>(gamma, c, ga + i * R::N);
#pragma unroll
            for (int e = 0; e < R::N; e++)
                o[e] = w.r * (fmaf(-xh[i * R::N + e], c2, g[e] * ga[i * R::N + e]) - c1);
            if (dsum) {
                float q[R::N];
                R::unpack(w.ds[i], q);
#pragma unroll
                for (int e = 0; e < R::N; e++) o[e] += q[e];
            }
            dx[base + c] = R::pack(o);
        }
    }
    if (!part) return;
    // the workgroup's rows together, in the order of their row slots
    const int64_t d = (int64_t)nv * R::N;
    float *pg = part + (int64_t)blockIdx.x * (RMS ? 1 : 2) * d, *pb = pg + d;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = lane + i * G;
#pragma unroll
        for (int z = 0; z < (RMS ? 1 : 2); z++) {
            float *a = (z ? db : dg) + i * R::N, *p = z ? pb : pg;
            if constexpr (G >= 256) {
                if (c < nv)
#pragma unroll
                    for (int e = 0; e < R::N; e += 4)
                        *reinterpret_cast<float4 *>(p + (int64_t)c * R::N + e) =
                            make_float4(a[e], a[e + 1], a[e + 2], a[e + 3]);
            } else {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < R::N; e++) acc_s[(threadIdx.x / G * R::N + e) * G + lane] = a[e];
                __syncthreads();
                // G * N columns, RPB terms each
                for (int m = threadIdx.x; m < G * R::N; m += 256) {
                    const int e = m % R::N, l = m / R::N;
                    float s = 0.f;
#pragma unroll
                    for (int b = 0; b < RPB; b++) s += acc_s[(b * R::N + e) * G + l];
                    if (l + i * G < nv) p[(int64_t)i * G * R::N + m] = s;
                }
            }
        }
    }
}

// dgamma, dbeta (gridDim.y = 2; 1: dgamma alone) = (+=) the workgroups' sums: 32 columns a workgroup, the sums
// dealt to 32 slices (16 loads of each in flight), the slices added in order.
// Bound by latency: 512 sums of 2 x 2048 columns (8.4 MB) in 4.6 us; one load at
// a time took 17 us.
__global__ __launch_bounds__(1024) void norm_bwd_params(const float *__restrict__ part, int np,
                                                        int d, float *__restrict__ dgamma,
                                                        float *__restrict__ dbeta, int accumulate) {
    __shared__ float s_p[32][33];
    const int z = blockIdx.y, nz = gridDim.y;
    float *out = z ? dbeta : dgamma;
    if (!out) return;
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
    const float *p = part + (int64_t)z * d + col;
    float s = 0.f;
    for (int i0 = sl; i0 < np; i0 += 32 * 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = i0 + 32 * i < np ? p[(int64_t)(i0 + 32 * i) * nz * d] : 0.f;
#pragma unroll
        for (int i = 0; i < 16; i++) s += v[i];
    }
    s_p[sl][threadIdx.x & 31] = s;
    __syncthreads();
    if (sl) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i++) s += s_p[i][threadIdx.x];
    out[col] = accumulate ? out[col] + s : s;
}

// ---------------------------------------------------------------------------
// launchers

// p + n elements of T, null if p is
template <typename E, typename P>
static E *at(P *p, int64_t n) { return p ? reinterpret_cast<E *>(p) + n : nullptr; }

// Threads of a row of nv vectors. One vector a thread is fastest where it
// keeps the threads busy (256 MiB of rows, forward: bf16 d = 2048 with 256 x 1
// 57 us, 64 x 4 72 us; d = 512 with 64 x 1 58 us, 32 x 2 62 us, 16 x 4 67 us), two
// or three where the next group would be mostly idle (forward d = 544: 64 x 2
// 67 us, 256 x 1 half of that filled; backward, which also pays for idle
// threads' registers, d = 320: 32 x 2 52 us, 64 x 1 60 us; d = 1280: 64 x 3 51
// us, 256 x 1 61 us). The backward stays below 1024 threads, where it has no
// registers to load ahead, up to three vectors a thread (bf16 d = 5120: 512 x 2
// 55 us, 1024 x 1 62 us).
constexpr int kNormGroups[] = {4, 8, 16, 32, 64, 256, 512, 1024};
constexpr int norm_group(int nv, bool bwd) {
    if (nv > (bwd ? 1536 : 1024)) return 1024;
    int i = 0;
    while (i < 7 && kNormGroups[i] < nv) i++;
    if (bwd && i == 7) return 512;
    return i > 0 && nv * 100 < kNormGroups[i] * (bwd ? 80 : 70) ? kNormGroups[i - 1] : kNormGroups[i];
}
constexpr int norm_vecs(int nv, bool bwd) {
    return (nv + norm_group(nv, bwd) - 1) / norm_group(nv, bwd);
}
constexpr bool norm_covered() {
    for (int nv = 4; nv <= 4096; nv += 4)
        if (norm_vecs(nv, false) > 4 || norm_vecs(nv, true) > 4) return false;
    return true;
}
static_assert(norm_covered(), "NORM_SWITCH has up to four vectors a thread");
// whether any width (d = 32, 64, ..) of the type uses G threads of V vectors
template <bool BF16>
constexpr bool norm_used(int g, int v, bool bwd) {
    for (int nv = 32 / Row16<BF16>::N; nv <= 16384 / Row16<BF16>::N; nv += 32 / Row16<BF16>::N)
        if (norm_group(nv, bwd) == g && norm_vecs(nv, bwd) == v) return true;
    return false;
}

// F(G, V) for the G and V of a row
#define NORM_IF(G, V, BWD, F)                            \
    if constexpr (norm_used<BF16>(G, V, BWD)) {          \
        if (g == G && v == V) { F(G, V); }               \
    }
#define NORM_IFS(G, BWD, F)                                                                  \
    NORM_IF(G, 1, BWD, F) NORM_IF(G, 2, BWD, F) NORM_IF(G, 3, BWD, F) NORM_IF(G, 4, BWD, F)
#define NORM_SWITCH(BWD, F)                                                                  \
    NORM_IFS(4, BWD, F) NORM_IFS(8, BWD, F) NORM_IFS(16, BWD, F) NORM_IFS(32, BWD, F)        \
    NORM_IFS(64, BWD, F) NORM_IFS(256, BWD, F) NORM_IFS(512, BWD, F) NORM_IFS(1024, BWD, F)

template <bool BF16, bool RMS>
static moe_status norm_fwd_run(const void *x, const void *res, const float *gamma,
                               const float *beta, float eps, int64_t T, int d, void *y, void *sum,
                               float *mean, float *rstd, uint8_t *x8, uint8_t *x8_scale,
                               uint8_t *yq, uint8_t *yq_scale, hipStream_t s) {
    typedef typename Codes<BF16>::type C;
    const int nv = d / Row16<BF16>::N, g = norm_group(nv, false), v = norm_vecs(nv, false);
    const int nt = norm_threads(g), rows = nt / g;
    typedef typename std::conditional<RMS, double, float>::type Inv;
    const Inv inv_d = (Inv)1 / (Inv)d;
    const int64_t piece = kMaxBlocks * rows;
    for (int64_t t = 0; t < T; t += piece) {
        const int64_t n = T - t < piece ? T - t : piece;
        const unsigned nb = (unsigned)((n + rows - 1) / rows);
        const int64_t o = t * nv;
#define F(G, V)                                                                                  \
    norm_fwd<BF16, G, V, RMS><<<nb, nt, 0, s>>>(                                                 \
        at<const uint4>(x, o), at<const uint4>(res, o), gamma, beta, eps, n, nv, inv_d,          \
        at<uint4>(y, o), at<uint4>(sum, o), at<float>(mean, t), at<float>(rstd, t), at<C>(x8, o), \
        at<uint8_t>(x8_scale, o / Row16<BF16>::LPB), at<C>(yq, o),                               \
        at<uint8_t>(yq_scale, o / Row16<BF16>::LPB))
        NORM_SWITCH(false, F)
#undef F
    }
    return launch_status();
}

moe_status norm_fwd_launch(const void *x, moe_dtype dt, const void *res, const float *gamma,
                           const float *beta, float eps, int64_t T, int d, void *y, void *sum,
                           float *mean, float *rstd, uint8_t *x8, uint8_t *x8_scale,
                           hipStream_t s) {
    return dt == MOE_BF16
               ? norm_fwd_run<true, false>(x, res, gamma, beta, eps, T, d, y, sum, mean, rstd, x8, x8_scale, nullptr, nullptr, s)
               : norm_fwd_run<false, false>(x, res, gamma, beta, eps, T, d, y, sum, mean, rstd, x8, x8_scale, nullptr, nullptr, s);
}

moe_status rms_fwd_launch(const void *x, moe_dtype dt, const void *res, const float *gamma,
                          float eps, int64_t T, int d, void *y, void *sum, float *rstd,
                          uint8_t *x8, uint8_t *x8_scale, uint8_t *yq, uint8_t *yq_scale,
                          hipStream_t s) {
    return dt == MOE_BF16
               ? norm_fwd_run<true, true>(x, res, gamma, nullptr, eps, T, d, y, sum, nullptr, rstd, x8, x8_scale, yq, yq_scale, s)
               : norm_fwd_run<false, true>(x, res, gamma, nullptr, eps, T, d, y, sum, nullptr, rstd, x8, x8_scale, yq, yq_scale, s);
}

// Workgroups of the backward, and rows of its partial sums: by the sizes
// alone, so that the workspace is the same on every device. Two a compute
// unit, but no more than an eighth of the rows, while there is one a compute
// unit: the partial sums are 8 bytes a column, written and read back, so T / 8
// workgroups move 2 T d bytes beside a bf16 backward's 6 T d (a third, from
// 2048 to 4096 rows; from a checkpoint two fifths). More rows make that less,
// as 1 / T; below 2048 rows the 256 workgroups' part is the larger the fewer
// rows there are.
static int64_t norm_bwd_blocks(int64_t T, int nv) {
    const int g = norm_group(nv, true), rpb = norm_threads(g) / g;
    const int64_t most = (T + rpb - 1) / rpb, few = most < 256 ? most : 256;
    const int64_t want = T / 8 < 512 ? T / 8 : 512;
    return want > few ? (want < most ? want : most) : few;
}

size_t norm_bwd_ws_bytes(moe_dtype dt, int64_t T, int d) {
    return (size_t)norm_bwd_blocks(T, d / (dt == MOE_BF16 ? 8 : 4)) * 2 * d * sizeof(float);
}
size_t rms_bwd_ws_bytes(moe_dtype dt, int64_t T, int d) { return norm_bwd_ws_bytes(dt, T, d) / 2; }

// Bytes of a matrix from which the RMS backward reads its rows past the
// last-level cache (256 MiB), where a part of them would only push out the rest.
// us, through the cache -> past it, bf16 d = 2048 with a stream gradient: directly
// behind its forward; behind work that leaves dy and dsum in the cache and x not,
// as a training step's does; called again on the same rows:
//   32 MiB  27.8 -> 30.5   32.1 -> 30.4   28.0 -> 30.8
//   40      34.5 -> 34.2   36.1 -> 35.6   32.9 -> 35.8
//   64      51.4 -> 50.3   49.6 -> 50.1   46.9 -> 52.2
//   72      64.8 -> 53.4   54.9 -> 54.4   54.5 -> 55.4
//   128    115.5 -> 92.1  116.8 -> 91.9  100.1 -> 90.7
// The first two at 32 and 40 MiB: without dsum 24.0 -> 27.2, 28.7 -> 26.3 and 30.0 ->
// 30.5, 33.0 -> 30.1; from a checkpoint 27.5 -> 28.8, 33.1 -> 31.2 and 34.6 -> 33.4,
// 39.3 -> 36.2; fp32 d = 4096 26.3 -> 28.9, 28.9 -> 28.6 and 39.2 -> 39.3, 41.8 -> 38.2.
// With none of the rows in the cache past it is faster at every size (8 MiB 18.3 ->
// 16.1, 64 MiB 83.5 -> 54.2). The layer norm's backward is without it, as it was.
constexpr int64_t kOnceBytes = 40 << 20;

template <bool BF16, bool RMS>
static moe_status norm_bwd_run(const void *dy, const void *x, const uint8_t *x8,
                               const uint8_t *x8_scale, const float *mean, const float *rstd,
                               const float *gamma, const void *dsum, int64_t T, int d, void *dx,
                               float *dgamma, float *dbeta, bool accumulate, float *part,
                               hipStream_t s) {
    typedef typename Codes<BF16>::type C;
    const int nv = d / Row16<BF16>::N, g = norm_group(nv, true), v = norm_vecs(nv, true);
    const int np = (int)norm_bwd_blocks(T, nv);
    const float inv_d = 1.f / (float)d;
    const bool once = T * nv * 16 >= kOnceBytes;
#define F3(G, V, K, O)                                                                            \
    norm_bwd<BF16, G, V, K, RMS, O><<<np, norm_threads(G), 0, s>>>(                              \
        at<const uint4>(dy, 0), at<const uint4>(x, 0), at<const C>(x8, 0), x8_scale, mean, rstd, \
        gamma, at<const uint4>(dsum, 0), T, nv, inv_d, at<uint4>(dx, 0), part)
#define F2(G, V, K) if (RMS && once) F3(G, V, K, RMS); else F3(G, V, K, false)
#define F(G, V) if (x8) { F2(G, V, true); } else { F2(G, V, false); }
    if (np > 0) { NORM_SWITCH(true, F) }
#undef F
#undef F2
#undef F3
    if (dgamma || dbeta)
        norm_bwd_params<<<dim3(d / 32, RMS ? 1 : 2), 1024, 0, s>>>(part, np, d, dgamma, dbeta, accumulate);
    return launch_status();
}

moe_status norm_bwd_launch(const void *dy, moe_dtype dt, const void *x, const uint8_t *x8,
                           const uint8_t *x8_scale, const float *mean, const float *rstd,
                           const float *gamma, const void *dsum, int64_t T, int d, void *dx,
                           float *dgamma, float *dbeta, bool accumulate, float *part,
                           hipStream_t s) {
    return dt == MOE_BF16
               ? norm_bwd_run<true, false>(dy, x, x8, x8_scale, mean, rstd, gamma, dsum, T, d, dx, dgamma, dbeta, accumulate, part, s)
               : norm_bwd_run<false, false>(dy, x, x8, x8_scale, mean, rstd, gamma, dsum, T, d, dx, dgamma, dbeta, accumulate, part, s);
}

moe_status rms_bwd_launch(const void *dy, moe_dtype dt, const void *x, const uint8_t *x8,
                          const uint8_t *x8_scale, const float *rstd, const float *gamma,
                          const void *dsum, int64_t T, int d, void *dx, float *dgamma,
                          bool accumulate, float *part, hipStream_t s) {
    return dt == MOE_BF16
               ? norm_bwd_run<true, true>(dy, x, x8, x8_scale, nullptr, rstd, gamma, dsum, T, d, dx, dgamma, nullptr, accumulate, part, s)
               : norm_bwd_run<false, true>(dy, x, x8, x8_scale, nullptr, rstd, gamma, dsum, T, d, dx, dgamma, nullptr, accumulate, part, s);
}

}  // namespace moe
