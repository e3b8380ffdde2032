// clip.hip -- the global norm of many gradients, and their clipping.
//
//   N = sqrt(sum_i sum_e g_i[e]^2),  out_i = g_i min(1, max_norm / (N + 1e-6)).
//
// The squares are formed and summed in fp64: every fp32 or bf16 value's square
// is a normal fp64 number, so nothing overflows or vanishes where the norm
// itself is representable, and the sum of billions of squares loses nothing.
// The order is fixed by the sizes alone (no atomics).
//
// A list's tensors are cut into chunks of 32 KiB, walked by a grid that fits
// the chip; the list travels in the kernel's arguments (kGradMax tensors a
// launch), so a call needs no table in device memory and can be captured.
// The bound is memory: one read for the norm, one read and one write to clip.
// 805 M fp32 gradients of two tensors (3.2 GB): norm 463 us (6.95 TB/s), then
// clipped into other tensors 1190 us (5.4 TB/s of reads and writes). 60 tensors of
// both types at odd addresses (21 MB) 18 us for both.
#include <type_traits>

#include "act8.h"
#include "common.h"

namespace moe {

constexpr int kGradMax = 64;            // tensors of a launch
constexpr int kChunkBytes = 32768;      // of a tensor: 8 vectors a thread
constexpr int kGradBlocks = 2048;       // workgroups of a launch: eight a compute unit

// A list of up to 16 pieces (of 1024 elements of one tensor) goes to one
// workgroup. It saves the host a launch (clipping 6.6 us a call and not 9.7, the
// norm 6.4 and 9.1) and is as fast on the GPU: clipping one tensor of 64 elements
// 3.4 us and 4.2, four of 1024 4.7 and 5.4, four of 4096 6.1 and 6.2, 16 of 1024
// 6.3 and 6.1; with 32 pieces it takes 9.1 to 10.1 us and not 5.5 to 6.4.
constexpr int kFewPiece = 1024, kFewPieces = 16;

struct GradItem {
    const char *in;
    char *out;
    int64_t n;          // elements
    int64_t first;      // chunks of the tensors in front of it
    int32_t bf16;
};
struct GradArgs {
    GradItem t[kGradMax];
    int64_t chunks;
    int32_t count;
};

// Vectors of 16 bytes at any element's address (the memory unit takes loads
// and stores that are not aligned to their size). ONCE: past the last-level
// cache, for what does not stay there until it is read again.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <bool ONCE>
MOE_DEV u32x4 load_any(const u32x4_any *p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool ONCE>
MOE_DEV void store_any(u32x4_any *p, const u32x4 &v) {
    if constexpr (ONCE) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// Chunks at a launch's end that the norm leaves in the last-level cache (256
// MiB, of which a list that is clipped into other tensors has half), and that
// the clipping, which walks a launch's chunks backwards, finds there. The others are
// read and written past it: 3.2 GB norm 520 -> 463 us, clipping 1240 -> 1165 us;
// 21 MB, all of which stays, 18.2 us for both and 20.3 past it. Those lists are one
// launch. Of a list of more than kGradMax tensors the launches go forwards in both
// passes and each keeps its own last chunks, most of which the next ones push out.
constexpr int64_t kGradKept = (128 << 20) / kChunkBytes;

template <bool BF16>
MOE_DEV float grad_elem(const char *p, int64_t i) {
    if constexpr (BF16) return bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
    else return reinterpret_cast<const float *>(p)[i];
}

// the last tensor of a list that starts at or before chunk c
MOE_DEV int tensor_of(const GradArgs &a, int64_t c) {
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.t[mid].first <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// f(tensor, first element, elements, whether the chunk is one of the launch's
// last kGradKept) for the chunks blockIdx.x, blockIdx.x + gridDim.x, .. of a
// launch; BACK: counted from its end.
template <bool BACK, typename F>
MOE_DEV void for_chunks(const GradArgs &a, F f) {
    for (int64_t i = blockIdx.x; i < a.chunks; i += gridDim.x) {
        const int64_t c = BACK ? a.chunks - 1 - i : i;
        const GradItem &t = a.t[tensor_of(a, c)];
        const int64_t per = t.bf16 ? kChunkBytes / 2 : kChunkBytes / 4;
        const int64_t e0 = (c - t.first) * per;
        const int64_t left = t.n - e0;
        f(t, e0, (int)(left < per ? left : per), c >= a.chunks - kGradKept);
    }
}

template <bool BF16, bool ONCE>
MOE_DEV double chunk_squares(const char *p, int64_t e0, int n) {
    typedef Row16<BF16> R;
    p += e0 * (BF16 ? 2 : 4);
    const int nv = n / R::N;
    double s[2] = {0., 0.};
    auto add = [&](const u32x4 &w) {
        float f[R::N];
        R::unpack(make_uint4(w.x, w.y, w.z, w.w), f);
#pragma unroll
        for (int e = 0; e < R::N; e++) {
            const double x = f[e];
            s[e & 1] = fma(x, x, s[e & 1]);
        }
    };
    const u32x4_any *v = reinterpret_cast<const u32x4_any *>(p);
    if (n == (BF16 ? kChunkBytes / 2 : kChunkBytes / 4)) {
        u32x4 w[8];
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = load_any<ONCE>(v + threadIdx.x + 256 * i);
#pragma unroll
        for (int i = 0; i < 8; i++) add(w[i]);
    } else {
        for (int i = threadIdx.x; i < nv; i += 256) add(v[i]);
        for (int i = nv * R::N + threadIdx.x; i < n; i += 256) {
            const double x = grad_elem<BF16>(p, i);
            s[0] = fma(x, x, s[0]);
        }
    }
    return s[0] + s[1];
}

// Sum over the workgroup's 256 threads, in a fixed order; all get it.
MOE_DEV double block_sum(double v) {
    __shared__ double w[4];
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = v;
    __syncthreads();
    return (w[0] + w[1]) + (w[2] + w[3]);
}

// part[blockIdx.x] = the sum of squares of the workgroup's chunks. A thread has 8
// vectors of a chunk in flight; the fp64 sums (a fused multiply-add an element)
// hide behind the reads.
__global__ __launch_bounds__(256) void grad_squares(GradArgs a, double *__restrict__ part) {
    double s = 0.;
    for_chunks<false>(a, [&](const GradItem &t, int64_t e0, int n, bool kept) {
        if (kept)
            s += t.bf16 ? chunk_squares<true, false>(t.in, e0, n) : chunk_squares<false, false>(t.in, e0, n);
        else
            s += t.bf16 ? chunk_squares<true, true>(t.in, e0, n) : chunk_squares<false, true>(t.in, e0, n);
    });
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// the partial sums' sum, by one workgroup's threads
MOE_DEV double sum_of(const double *part, int np) {
    double s = 0.;
    for (int i = threadIdx.x; i < np; i += 256) s += part[i];
    return block_sum(s);
}

// the norm from up to 2048 partial sums of each launch: 5 us, a chain of latencies.
// Their sum takes the place of the first of them, for a clipping behind it.
__global__ __launch_bounds__(256) void grad_finish(double *part, int np, float *__restrict__ norm) {
    const double s = sum_of(part, np);
    if (threadIdx.x == 0) {
        *norm = (float)sqrt(s);
        part[0] = s;
    }
}

// A norm beyond fp32's range is infinite here as it is to the caller: a clipping
// by the norm that was returned has the same factor, 0.
MOE_DEV float clip_scale(double norm, float max_norm) {
    if (__builtin_isinf((float)norm)) return 0.f;
    const double q = (double)max_norm / (norm + 1e-6);
    return q >= 1. ? 1.f : (float)q;             // a NaN stays one
}

template <bool BF16, bool ONCE>
MOE_DEV void chunk_scale(const GradItem &t, int64_t e0, int n, float scale) {
    typedef Row16<BF16> R;
    constexpr int S = BF16 ? 2 : 4;
    const char *p = t.in + e0 * S;
    char *o = t.out + e0 * S;
    const int nv = n / R::N;
    const u32x4_any *v = reinterpret_cast<const u32x4_any *>(p);
    u32x4_any *q = reinterpret_cast<u32x4_any *>(o);
    auto scaled = [&](const u32x4 &w) {
        float f[R::N];
        R::unpack(make_uint4(w.x, w.y, w.z, w.w), f);
#pragma unroll
        for (int e = 0; e < R::N; e++) f[e] *= scale;
        const uint4 r = R::pack(f);
        return u32x4{r.x, r.y, r.z, r.w};
    };
    if (n == kChunkBytes / S) {
        u32x4 w[8];
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = load_any<ONCE>(v + threadIdx.x + 256 * i);
#pragma unroll
        for (int i = 0; i < 8; i++) store_any<ONCE>(q + threadIdx.x + 256 * i, scaled(w[i]));
    } else {
        for (int i = threadIdx.x; i < nv; i += 256) q[i] = scaled(v[i]);
        for (int i = nv * R::N + threadIdx.x; i < n; i += 256) {
            const float x = grad_elem<BF16>(p, i) * scale;
            if constexpr (BF16) reinterpret_cast<uint16_t *>(o)[i] = f32_to_bf16(x);
            else reinterpret_cast<float *>(o)[i] = x;
        }
    }
}

// out = in * scale; the scale from the partial sums (part; workgroup 0 then
// leaves the norm) or from *norm. A scale of one leaves tensors that are
// written in place as they are. The product is rounded to fp32 and from there to
// the output's type (bf16: at most 2^-24 of the value beyond half a step). Every
// workgroup adds the partial sums itself, from the last-level cache, in the same
// order: a launch for them alone costs 5 us and another gap.
__global__ __launch_bounds__(256) void grad_scale(GradArgs a, const double *__restrict__ part,
                                                  int np, float *__restrict__ norm,
                                                  float max_norm) {
    double v;
    if (part) {
        v = sqrt(sum_of(part, np));
        if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
    } else {
        v = *norm;
    }
    const float scale = clip_scale(v, max_norm);
    const bool once = a.chunks > kGradKept;
    for_chunks<true>(a, [&](const GradItem &t, int64_t e0, int n, bool) {
        if (scale == 1.f && t.in == t.out) return;
        if (once) {
            if (t.bf16) chunk_scale<true, true>(t, e0, n, scale);
            else chunk_scale<false, true>(t, e0, n, scale);
        } else {
            if (t.bf16) chunk_scale<true, false>(t, e0, n, scale);
            else chunk_scale<false, false>(t, e0, n, scale);
        }
    });
}

// The whole of a short list in one workgroup and one launch: a wave has one
// piece of it, which stays in registers from the norm to the clipping. Bound by
// latency (3.4 to 6 us); rounded as in grad_scale.
__global__ __launch_bounds__(1024) void grad_clip_few(GradArgs a, float *__restrict__ norm,
                                                      float max_norm, int clip) {
    __shared__ double w[16];
    constexpr int L = kFewPiece / 64;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool mine = wave < a.chunks;
    const GradItem &t = a.t[mine ? tensor_of(a, wave) : 0];
    const int64_t e0 = (wave - t.first) * kFewPiece;
    const int n = mine ? (int)min(t.n - e0, (int64_t)kFewPiece) : 0;
    float v[L];
    double s = 0.;
    if (mine) {
        auto read = [&](auto bf16) {
#pragma unroll
            for (int i = 0; i < L; i++) v[i] = grad_elem<decltype(bf16)::value>(t.in, e0 + min(lane + 64 * i, n - 1));
        };
        if (t.bf16) read(std::true_type{});
        else read(std::false_type{});
#pragma unroll
        for (int i = 0; i < L; i++) {
            const double x = lane + 64 * i < n ? v[i] : 0.f;
            s = fma(x, x, s);
        }
    }
    s = wave_sum(s);
    if (lane == 0) w[wave] = s;
    __syncthreads();
    s = 0.;
#pragma unroll
    for (int i = 0; i < 16; i++) s += w[i];
    const double all = sqrt(s);
    if (threadIdx.x == 0) *norm = (float)all;
    if (!clip || !mine) return;
    const float scale = clip_scale(all, max_norm);
    if (scale == 1.f && t.in == t.out) return;
#pragma unroll
    for (int i = 0; i < L; i++) {
        const int64_t e = e0 + lane + 64 * i;
        if (lane + 64 * i >= n) break;
        if (t.bf16) reinterpret_cast<uint16_t *>(t.out)[e] = f32_to_bf16(v[i] * scale);
        else reinterpret_cast<float *>(t.out)[e] = v[i] * scale;
    }
}

// ---------------------------------------------------------------------------
// launchers

// The next launch's tensors of a list from item i on (empty ones left out);
// returns the item after them. few: cut for grad_clip_few.
static int grad_args(const moe_grad *g, int n, int i, GradArgs &a, bool few = false) {
    a.count = 0;
    a.chunks = 0;
    for (; i < n && a.count < kGradMax; i++) {
        if (g[i].n == 0) continue;
        const int per = few ? kFewPiece : kChunkBytes / (g[i].dtype == MOE_BF16 ? 2 : 4);
        GradItem &t = a.t[a.count++];
        t.in = (const char *)g[i].data;
        t.out = (char *)(g[i].out ? g[i].out : g[i].data);
        t.n = g[i].n;
        t.first = a.chunks;
        t.bf16 = g[i].dtype == MOE_BF16;
        a.chunks += (g[i].n + per - 1) / per;
    }
    return i;
}

static unsigned grad_blocks(const GradArgs &a) {
    return (unsigned)(a.chunks < kGradBlocks ? a.chunks : kGradBlocks);
}

size_t grad_norm_ws_bytes(int n) {
    return (size_t)((n + kGradMax - 1) / kGradMax) * kGradBlocks * sizeof(double);
}

// the partial sums of a list; their number
static int grad_squares_launch(const moe_grad *g, int n, double *part, hipStream_t s) {
    int np = 0;
    GradArgs a;
    for (int i = 0; i < n;) {
        i = grad_args(g, n, i, a);
        if (a.count == 0) break;
        const unsigned nb = grad_blocks(a);
        grad_squares<<<nb, 256, 0, s>>>(a, part + np);
        np += (int)nb;
    }
    return np;
}

// Whether the list is one for grad_clip_few: a then holds all of it.
static bool grad_few(const moe_grad *g, int n, GradArgs &a) {
    int64_t pieces = 0;
    for (int i = 0; i < n && pieces <= kFewPieces; i++) pieces += (g[i].n + kFewPiece - 1) / kFewPiece;
    return pieces <= kFewPieces && grad_args(g, n, 0, a, true) == n;
}

moe_status grad_norm_launch(const moe_grad *g, int n, float *norm, void *ws, hipStream_t s) {
    GradArgs a;
    if (grad_few(g, n, a)) {
        grad_clip_few<<<1, 1024, 0, s>>>(a, norm, 0.f, 0);
        return launch_status();
    }
    const int np = grad_squares_launch(g, n, (double *)ws, s);
    grad_finish<<<1, 256, 0, s>>>((double *)ws, np, norm);
    return launch_status();
}

moe_status grad_clip_launch(const moe_grad *g, int n, float max_norm, float *norm, void *ws,
                            hipStream_t s) {
    const double *part = nullptr;
    int np = 0;
    GradArgs a;
    if (ws && grad_few(g, n, a)) {
        grad_clip_few<<<1, 1024, 0, s>>>(a, norm, max_norm, 1);
        return launch_status();
    }
    if (ws) {
        np = grad_squares_launch(g, n, (double *)ws, s);
        // few partial sums: every workgroup adds them itself
        if (np > kGradBlocks) {
            grad_finish<<<1, 256, 0, s>>>((double *)ws, np, norm);
            np = 1;
        }
        part = (const double *)ws;
    }
    for (int i = 0; i < n;) {
        i = grad_args(g, n, i, a);
        if (a.count == 0) break;
        grad_scale<<<grad_blocks(a), 256, 0, s>>>(a, part, np, norm, max_norm);
    }
    return launch_status();
}

}  // namespace moe
