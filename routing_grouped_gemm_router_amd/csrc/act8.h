// act8.h -- 8-bit activation checkpoints on the device: the OCP MXINT8
// encoding and decoding steps (Open Compute Project Microscaling v1.0), shared
// by the checkpoint kernels (act8.hip) and the layer norm (norm.hip).
//
// A block of 32 neighbouring elements of a row has one E8M0 scale byte, e =
// the biased fp32 exponent of its largest magnitude, so 2^(e-127) <= amax <
// 2^(e-126) (fp32 subnormals and zero: e = 0), and 32 whole numbers
//   c = clamp(rne(x * 2^(133-e)), -127, 127)   standing for   c * 2^(e-133).
// The step 2^(e-133) is amax's power of two over 64, so an element is off by
// at most half a step (amax / 128); only the topmost half step, magnitudes
// beyond 127.5 steps, is off by up to one (the symmetric clamp). That is a
// uniform error where E4M3's is relative (2^-4 of each element): for the same
// byte, the largest elements of a block, which dominate a gradient's sums,
// keep 7 bits instead of 3.
// A block holding a NaN or an infinity gets e = 255 (E8M0's NaN) and zeros,
// and is restored as 32 NaNs: an overflow stays visible in the gradients.
// Every other value is exactly representable in bf16: 7 significant bits,
// and the smallest step, 2^-133, is bf16's smallest subnormal.
#pragma once

#include "common.h"

namespace moe {

// A grid has fewer than 2^32 threads: at most 2^21 workgroups (of up to 1024)
// a launch, larger inputs in pieces.
constexpr int64_t kMaxBlocks = 1 << 21;

// 16-byte vectors of a row: 8 bf16 or 4 fp32 elements
template <bool BF16>
struct Row16 {
    static constexpr int N = BF16 ? 8 : 4;        // elements of a vector
    static constexpr int LPB = 32 / N;            // lanes (vectors) of a block of 32
    MOE_DEV static void unpack(const uint4 &v, float *f) {
        if constexpr (BF16) {
            f[0] = lo_bf16(v.x); f[1] = hi_bf16(v.x); f[2] = lo_bf16(v.y); f[3] = hi_bf16(v.y);
            f[4] = lo_bf16(v.z); f[5] = hi_bf16(v.z); f[6] = lo_bf16(v.w); f[7] = hi_bf16(v.w);
        } else {
            f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
            f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
        }
    }
    MOE_DEV static uint4 pack(const float *f) {
        uint4 v;
        if constexpr (BF16) {
            v.x = pack_bf16x2(f[0], f[1]); v.y = pack_bf16x2(f[2], f[3]);
            v.z = pack_bf16x2(f[4], f[5]); v.w = pack_bf16x2(f[6], f[7]);
        } else {
            v.x = __float_as_uint(f[0]); v.y = __float_as_uint(f[1]);
            v.z = __float_as_uint(f[2]); v.w = __float_as_uint(f[3]);
        }
        return v;
    }
};

// The codes of one vector: 8 bytes (bf16) or 4 (fp32).
template <bool BF16> struct Codes;
template <> struct Codes<true> { typedef uint2 type; };
template <> struct Codes<false> { typedef uint32_t type; };

// Loads of what this kernel reads once and nobody reads soon again, stores
// likewise: they leave the last-level cache to the others.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
MOE_DEV uint4 load_once(const uint4 *p) {
    const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
    return make_uint4(w.x, w.y, w.z, w.w);
}
MOE_DEV uint2 load_once(const uint2 *p) {
    const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
    return make_uint2(w.x, w.y);
}
MOE_DEV uint32_t load_once(const uint32_t *p) { return __builtin_nontemporal_load(p); }
MOE_DEV void store_once(uint4 *p, const uint4 &v) {
    __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4 *>(p));
}
MOE_DEV void store_once(uint2 *p, const uint2 &v) {
    __builtin_nontemporal_store(u32x2{v.x, v.y}, reinterpret_cast<u32x2 *>(p));
}
MOE_DEV void store_once(uint32_t *p, uint32_t v) { __builtin_nontemporal_store(v, p); }

MOE_DEV uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The scale byte of the block that this lane's vector belongs to: the
// magnitudes' bit patterns are compared as integers (NaN above infinity above
// every finite value), first within the vector, then over the block's 4
// (bf16) or 8 (fp32) neighbouring lanes. All lanes of the block must be
// active, and the first of them a multiple of the block's lane count.
template <bool BF16>
MOE_DEV uint32_t act8_scale_byte(const uint4 &v) {
    uint32_t m;
    if constexpr (BF16) {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        auto half = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7fff7fffu); };
        const u16x2 p = __builtin_elementwise_max(__builtin_elementwise_max(half(v.x), half(v.y)),
                                                  __builtin_elementwise_max(half(v.z), half(v.w)));
        m = umax(p.x, p.y);
    } else {
        const uint32_t k = 0x7fffffffu;
        m = umax(umax(v.x & k, v.y & k), umax(v.z & k, v.w & k));
    }
    m = umax(m, (uint32_t)dpp_move<kDppXor1>((int)m));
    m = umax(m, (uint32_t)dpp_move<kDppXor2>((int)m));
    if constexpr (!BF16) m = umax(m, (uint32_t)dpp_move<kDppHalfMirror>((int)m));
    return BF16 ? m >> 7 : m >> 23;
}

// Four elements to their four bytes (first lowest), scale byte sb. Adding
// 1.5 * 2^23 rounds to nearest even and leaves the whole number, two's
// complement, in the low bits.
MOE_DEV uint32_t act8_encode4(float a, float b, float c, float d, uint32_t sb) {
    const float x[4] = {a, b, c, d};
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float t = __builtin_amdgcn_fmed3f(ldexpf(x[i], 133 - (int)sb), -127.f, 127.f);
        u[i] = __float_as_uint(t + 12582912.f);
    }
    const uint32_t lo = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(u[3], u[2], 0x0c0c0400u);
    const uint32_t w = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    return sb == 255 ? 0u : w;
}

MOE_DEV void act8_encode(const float *f, uint32_t sb, uint2 &q) {
    q.x = act8_encode4(f[0], f[1], f[2], f[3], sb);
    q.y = act8_encode4(f[4], f[5], f[6], f[7], sb);
}
MOE_DEV void act8_encode(const float *f, uint32_t sb, uint32_t &q) {
    q = act8_encode4(f[0], f[1], f[2], f[3], sb);
}

// The step that scale byte sb stands for (NaN for 255).
MOE_DEV float act8_step(uint32_t sb) {
    return sb == 255 ? __builtin_nanf("") : ldexpf(1.f, (int)sb - 133);
}

// Four bytes to the values they stand for: exact, c * step has 7 bits.
MOE_DEV void act8_decode4(uint32_t w, float step, float *f) {
    f[0] = (float)(int8_t)w * step;
    f[1] = (float)(int8_t)(w >> 8) * step;
    f[2] = (float)(int8_t)(w >> 16) * step;
    f[3] = (float)(int8_t)(w >> 24) * step;
}
MOE_DEV void act8_decode(const uint2 &q, float step, float *f) {
    act8_decode4(q.x, step, f);
    act8_decode4(q.y, step, f + 4);
}
MOE_DEV void act8_decode(const uint32_t &q, float step, float *f) { act8_decode4(q, step, f); }

// silu(a) = a sigmoid(a), from E = exp(-|a| / 2): E^2 / (1 + E^2) for a < 0,
// 1 / (1 + E^2) otherwise. exp(-a) itself would overflow below a = -88 and
// lose the product a exp(a) where it is still a normal number.
MOE_DEV float silu(float a) {
    const float e = expf(-0.5f * fabsf(a));
    return (a < 0.f ? (a * e) * e : a) / fmaf(e, e, 1.f);
}

}  // namespace moe
