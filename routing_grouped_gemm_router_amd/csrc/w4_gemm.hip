// w4_gemm.hip -- grouped products of MXFP8 rows with MXFP4 weights, and the
// experts' forward of a prompt built on them.
//
//   C[r, n] = sum_k A[src(r), k] B[e(r)][n, k],  src(r) = a_rows[r] or r,
// E4M3 elements on the left, E2M1 on the right, both with an E8M0 scale per 32
// along k, in v_mfma_scale_f32_32x32x64_f8f6f4 with fp32 sums. The instruction
// takes the two formats as they are stored and runs at the rate of E4M3 (4.6
// PFLOP/s in a loop of nothing else on this card, 8x8 and 8x4 alike): 4-bit
// weights halve what is read of them, from HBM and from LDS.
//
// The weights are the instruction's first operand, the rows its second, so
// that a lane holds 16 of 32 neighbouring outputs n of one row: two lanes hold
// a 32-element block of H', whose scale is one exchange away, and the outputs
// leave in 16-byte pieces after one 32-lane swap a register.
//
// Tiles, schedule and copies into LDS as in the grouped GEMM (gemm_device.h):
// a persistent grid walks each expert's tiles, an XCD its own weight panels.
// Every wave copies and multiplies; two workgroups a compute unit cover each
// other's barriers and epilogues. A step is 128 of K: 128 bytes of each row, 64
// of each weight row, four scales of each. Where a row's scales come in whole 16
// bytes (K a multiple of 512) those of four steps are copied together and read from
// LDS once, into two registers a row from which the instruction picks its byte (up,
// K = N = 2048, 8 experts of 256 rows 19.6 -> 17.9 us against a read a step, 65536 rows
// of 128 experts 280 -> 272). H' is rounded once, from fp32 to the MXFP8 that the
// second product multiplies; the prompt's y once, to fp16 of a block's own scale
// (kOutHalf): rounded to bf16 it would cost the output as much as out's own rounding
// (2.5e-3 from 64 bits in the 2-norm and not 1.8e-3), for 1 % of the time. Of those
// 1.8e-3 out's rounding is 1.66e-3; the rest is H' on another E4M3 code than the exact
// value's, 7 elements in 10,000, from the matrix unit's sums (off by some 4.4e-6 of their
// rms; the fp32 SwiGLU adds 1 in 10 million).
//
// 65536 rows, up and down: E = 128, d = 2048, h = 1024 270 and 174 us (2.0 and
// 1.58 PFLOP/s); E = 8, d = 4096, h = 2048 900 and 510 us (2.45 and 2.15). Of E =
// 128's up (279 us in that run) the copies and outputs alone take 235 us (64-byte
// weight rows cost the L1 a whole line each), the copies 203, products, LDS reads and
// outputs without copies 221 (on random data the chip's power holds the clock at 1.9
// GHz); of its down (177) the copies and outputs 175, the copies 87, copies and
// products without outputs 121: a tile's outputs come all at once.
#include <type_traits>

#include "act8.h"
#include "common.h"
#include "copy_plan.h"
#include "gemm_device.h"
#include "mx_encode.h"

namespace moe {

// Rows of 64 bytes in LDS: four lie in one sweep of the 64 banks, so the
// 16-byte pieces are swizzled by (row / 4) % 4, which puts the 16 rows that a
// ds_read_b128 serves at once on 16 different bank groups.
MOE_DEV int w4_chunk(int row, int c) { return row * 4 + (c ^ ((row >> 2) & 3)); }

// Chunks of the schedule, at least: two an XCD. One an XCD is as good with 8
// groups alike (K = N = 2048: within 2 %), with unlike ones worse (2048 rows of 8
// groups, N = 8192, K = 4096, small tiles: 200 us where no chunk is cut, 199 with 8,
// 182 with 16, 185 with 32, 190 with 64). 2 groups of 512 rows, K = N = 8192, large
// tiles: 213 us where none is cut, 85 with 16.
constexpr int kUnits = 16;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
MOE_DEV uint32_t pack_f16x2(float a, float b) { return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b}); }

struct W4GemmTile {
    int e, row0, row_end, nt;
};

// What a tile's sums become. kOutHidden: the weight rows of a wave are gate rows,
// then the up rows of the same hidden units; c is E4M3 H' [rows, N / 2] with c_scale.
// kOutBf16: c is bf16 [rows, N]. kOutHalf: c is fp16 [rows, N], per 32 columns times
// 2^(c_scale - 127): 11 significant bits or more of what counts in a block, in the
// bytes of bf16 and one more in 64.
enum { kOutBf16, kOutHidden, kOutHalf };

// BM rows x BN weight rows a tile, WM x WN waves.
template <int OUT, bool BATCHED, int BM, int BN, int WM, int WN, int STAGES, int OCC>
__global__ __launch_bounds__(WM *WN * 64) __attribute__((amdgpu_waves_per_eu(OCC, OCC)))
void w4_gemm_tiles(moe_w4_gemm_desc g) {
    constexpr bool SWIGLU = OUT == kOutHidden;
    constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
    static_assert(!SWIGLU || TN % 2 == 0, "gate and up of a unit in one wave");
    static_assert(NW * 64 >= 256, "the tile table's scan");
    // Weights in whole 128-byte lines, of two steps, where LDS has room for two such
    // (the L1 takes a whole line's time for the 64 bytes of one step; K = N = 2048,
    // small tiles: 128 experts of 32 rows 57.6 -> 54.5 us, medium ones: 2 experts of 512
    // rows, K = N = 8192, 65.9 -> 62.9; 8 experts of 32 rows 10.6 -> 10.9)
    constexpr bool LINES = BATCHED && BN <= 128;
    constexpr int BP = LINES ? 8 : 4;                                 // 16-byte pieces of a weight row
    constexpr int IPA = BM * 8 / 64 / NW, IPB = BN * BP / 64 / NW;    // 16-byte copies a lane
    static_assert(IPA * 64 * NW == BM * 8 && IPB * 64 * NW == BN * BP, "whole copies");
    constexpr int SROWS = BM + BN, SPW = (SROWS / 64 + NW - 1) / NW;  // scale words
    static_assert(BM % 64 == 0 && BN % 64 == 0, "a wave's scale words are of one operand");
    static_assert(STAGES == 2 || STAGES == 3, "two slots of four steps of scales");
    constexpr int AST = BM * 8, BST = BN * BP, BSTAGES = LINES ? 2 : STAGES;   // uint4
    constexpr int POOL = STAGES * AST + BSTAGES * BST;
    static_assert(!LINES || STAGES <= 3, "a line's place is free again when the next but one is copied");
    // the grid has as many workgroups as fit: LDS with the tables' 4.1 KiB
    static_assert((POOL + 2 * SROWS) * 16 + 4048 <= 163840 / (OCC * 4 / NW), "LDS");
    __shared__ __attribute__((aligned(1024))) uint4 pool[POOL];
    // scale words: a slot for each stage, 4 bytes a row, or where a row's scales
    // come in whole 16-byte groups two slots of four steps
    __shared__ __attribute__((aligned(1024))) uint4 scales[2 * SROWS];
    __shared__ int32_t s_off[257], s_tile[257], s_chunk[257], s_xpre[kXcdChunks + 1];

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int E = g.n_groups, K = g.K, N = g.N, h = N / 2;
    const int xcd = blockIdx.x & 7, workers = gridDim.x >> 3;
    build_tile_table(g.offsets, E, BM, s_off, s_tile);
    const int n_tiles = SWIGLU ? (h + BN / 2 - 1) / (BN / 2) : (N + BN - 1) / BN;
    const RowSchedule rs = build_row_schedule(s_tile, E, n_tiles, xcd, s_chunk, s_xpre, kUnits);
    const int nk = K / 128;

    // weight row (of N) of the tile's row n, the last one past the end
    auto b_row = [&](int nt, int n) {
        if constexpr (SWIGLU) {
            constexpr int HW = WTN / 2;
            const int o = n % WTN, j = min(nt * (BN / 2) + n / WTN * HW + o % HW, h - 1);
            return o < HW ? j : h + j;
        } else {
            return min(nt * BN + n, N - 1);
        }
    };
    auto decode = [&](int pos) {
        W4GemmTile t;
        int mt;
        decode_row_tile(rs, s_tile, s_chunk, s_xpre, E, xcd, pos, t.e, mt, t.nt);
        t.row0 = s_off[t.e] + mt * BM;
        t.row_end = s_off[t.e + 1];
        return t;
    };

    // the copies: this lane's sources of tile ipos, whose step ikt is the next
    const uint8_t *pa[IPA], *ps[SPW];
    uint32_t ob[IPB];
    const char *pb = nullptr;
    int ipos = blockIdx.x >> 3, ikt = 0, issued = 0, slot = 1;
    W4GemmTile ahead{};                  // the tile set up last
    auto setup = [&](const W4GemmTile &t) {
        // row r of the tile in A; past the group's end its last row
        auto src = [&](int r) {
            const int gr = min(t.row0 + r, t.row_end - 1);
            return (int64_t)(g.a_rows ? g.a_rows[gr] : gr);
        };
#pragma unroll
        for (int i = 0; i < IPA; i++) {
            const int p = (wave * IPA + i) * 64 + lane, r = p >> 3;
            pa[i] = g.a + src(r) * K + ((p & 7) ^ kl_swz(r)) * 16;
        }
        pb = uniform_ptr(reinterpret_cast<const char *>(g.b) + (int64_t)t.e * N * (K / 2));
#pragma unroll
        for (int i = 0; i < IPB; i++) {
            const int p = (wave * IPB + i) * 64 + lane, r = p / BP;
            ob[i] = (uint32_t)b_row(t.nt, r) * (uint32_t)(K / 2) +
                    ((p % BP) ^ (LINES ? kl_swz(r) : (r >> 2) & 3)) * 16;
        }
#pragma unroll
        for (int q = 0; q < SPW; q++) {
            const int s0 = (q * NW + wave) * 64;                  // wave-uniform
            if (s0 < BM) ps[q] = g.a_scale + src(s0 + lane) * (K / 32);
            else if (s0 < SROWS)
                ps[q] = g.b_scale + ((int64_t)t.e * N + b_row(t.nt, s0 + lane - BM)) * (K / 32);
        }
    };
    // enqueue the next step's copies, if there is one, into stage buf
    auto issue = [&](int buf, auto phase) {
        // BATCHED: the step of its four, known here; else any
        constexpr int P = decltype(phase)::value;
        if (ipos >= rs.total) return;
        if ((!BATCHED || P == 0) && ikt == 0) {
            ahead = decode(ipos);
            setup(ahead);
        }
        // scales first: a wait for the step's operands then covers them
        if constexpr (!BATCHED) {
#pragma unroll
            for (int q = 0; q < SPW; q++)
                if ((q * NW + wave) * 64 < SROWS)
                    dma4(ps[q] + ikt * 4, scales + buf * (SROWS / 4) + (q * NW + wave) * 16);
        } else if constexpr (P == 0) {
            slot ^= 1;
#pragma unroll
            for (int q = 0; q < SPW; q++)
                if ((q * NW + wave) * 64 < SROWS)
                    dma16(ps[q] + ikt * 4, scales + slot * SROWS + (q * NW + wave) * 64);
        }
        if (!LINES || (P & 1) == 0) {
            uint4 *bt = pool + STAGES * AST + (LINES ? P >> 1 : buf) * BST;
#pragma unroll
            for (int i = 0; i < IPB; i++) dma16s(ob[i], pb + ikt * 64, bt + (wave * IPB + i) * 64);
        }
#pragma unroll
        for (int i = 0; i < IPA; i++) dma16(pa[i] + ikt * 128, pool + buf * AST + (wave * IPA + i) * 64);
        issued++;
        ikt++;
        if ((!BATCHED || P == 3) && ikt == nk) {
            ikt = 0;
            ipos += workers;
        }
    };

    f32x16 acc[TN][TM];
    // rows r0 .. r0 + 31 of the stage, K slice s (64 wide): K 16 half .. + 15 of
    // the slice in dwords 0-3, 32 + 16 half .. + 15 in dwords 4-7; weights: K 32
    // half .. + 31 in dwords 0-3 (both layouts measured on the GPU)
    auto frag_a = [&](const uint4 *st, int r0, int s) {
        const int row = r0 + (lane & 31);
        const uint4 c0 = st[kl_chunk(row, 4 * s + half)], c1 = st[kl_chunk(row, 4 * s + 2 + half)];
        return i32x8{(int)c0.x, (int)c0.y, (int)c0.z, (int)c0.w, (int)c1.x, (int)c1.y, (int)c1.z, (int)c1.w};
    };
    auto frag_b = [&](const uint4 *st, int r0, int s) {
        const int row = r0 + (lane & 31);
        const uint4 c = st[LINES ? kl_chunk(row, 2 * s + half) : w4_chunk(row, 2 * s + half)];
        return i32x8{(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
    };
    // Scale bytes of this lane's rows: for slice s of a step the byte half + 2 s of
    // the row's word. BATCHED: those of four steps in two registers a row, which
    // the instruction picks by itself; else of one step.
    constexpr int SW = BATCHED ? 2 : 1;
    uint32_t sa[TM][SW], sb[TN][SW];
    auto read_scale = [&](int slot, int r, uint32_t (&o)[SW]) {
        if constexpr (BATCHED) {
            const uint4 w = scales[slot * SROWS + r];
            const uint32_t sel = half ? 0x07050301 : 0x06040200;
            o[0] = __builtin_amdgcn_perm(w.y, w.x, sel);
            o[1] = __builtin_amdgcn_perm(w.w, w.z, sel);
        } else {
            o[0] = reinterpret_cast<const uint32_t *>(scales)[slot * SROWS + r] >> (8 * half);
        }
    };
    auto read_scales = [&](int slot) {
#pragma unroll
        for (int i = 0; i < TM; i++) read_scale(slot, wm * WTM + i * 32 + (lane & 31), sa[i]);
#pragma unroll
        for (int j = 0; j < TN; j++) read_scale(slot, BM + wn * WTN + j * 32 + (lane & 31), sb[j]);
    };
    auto compute = [&](int buf, auto step_of_four) {
        constexpr int Q = decltype(step_of_four)::value;
        constexpr int W = BATCHED ? Q >> 1 : 0, S0 = BATCHED ? 2 * (Q & 1) : 0, S1 = BATCHED ? S0 + 1 : 2;
        const uint4 *st = pool + buf * AST, *bt = pool + STAGES * AST + (LINES ? Q >> 1 : buf) * BST;
        constexpr int B0 = LINES ? 2 * (Q & 1) : 0;      // the step's first slice in bt
        i32x8 fa[2][TM], fb[TN];
#pragma unroll
        for (int j = 0; j < TN; j++) fb[j] = frag_b(bt, wn * WTN + j * 32, B0);
#pragma unroll
        for (int i = 0; i < TM; i++) fa[0][i] = frag_a(st, wm * WTM + i * 32, 0);
        // the reads of slice 1 between the products of slice 0; a weight fragment
        // takes the place of the one whose products have just been issued
#pragma unroll
        for (int j = 0; j < TN; j++) {
#pragma unroll
            for (int i = 0; i < TM; i++) {
                __builtin_amdgcn_sched_barrier(0);
                acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    fb[j], fa[0][i], acc[j][i], 4, 0, S0, (int)sb[j][W], S0, (int)sa[i][W]);
                __builtin_amdgcn_sched_barrier(0);
                if (j * TM + i < TM) fa[1][j * TM + i] = frag_a(st, wm * WTM + (j * TM + i) * 32, 1);
            }
            fb[j] = frag_b(bt, wn * WTN + j * 32, B0 + 1);
        }
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int i = 0; i < TM; i++)
                acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    fb[j], fa[1][i], acc[j][i], 4, 0, S1, (int)sb[j][W], S1, (int)sa[i][W]);
    };
    // acc[j][i][4 q + x]: row i * 32 + lane % 32 of the wave, output j * 32 + 8 q +
    // 4 half + x. v_permlane32_swap gives the lower half of the lanes both
    // halves' values of one register and the upper half the other's.
    auto swap32 = [](uint32_t lo, uint32_t up, uint32_t &first, uint32_t &second) {
        const auto r = __builtin_amdgcn_permlane32_swap(lo, up, false, false);
        first = r[0];
        second = r[1];
    };
    // H' of the wave's tile in acc[j < TN / 2] to E4M3, by encode
    auto store_hidden = [&](const W4GemmTile &t, auto encode) {
#pragma unroll
        for (int i = 0; i < TM; i++) {
            const int row = t.row0 + wm * WTM + i * 32 + (lane & 31);
            uint8_t *c = reinterpret_cast<uint8_t *>(g.c) + (int64_t)row * h;
#pragma unroll
            for (int j = 0; j < TN / 2; j++) {
                const int n = t.nt * (BN / 2) + wn * (WTN / 2) + j * 32;
                if (n >= h) continue;                             // wave-uniform
                const f32x16 &f = acc[j][i];
                float am = 0.f;
#pragma unroll
                for (int v = 0; v < 16; v++) am = fmaxf(am, fabsf(f[v]));
                const uint32_t sb = mx_scale_byte(max_xor32(am));
                uint32_t w[4], o[4];
#pragma unroll
                for (int q = 0; q < 4; q++) w[q] = encode(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3], sb);
                swap32(w[0], w[2], o[0], o[1]);
                swap32(w[1], w[3], o[2], o[3]);
                if (row < t.row_end) {
                    *reinterpret_cast<uint4 *>(c + n + 16 * half) = make_uint4(o[0], o[1], o[2], o[3]);
                    if (half == 0) g.c_scale[(int64_t)row * (h / 32) + n / 32] = (uint8_t)sb;
                }
            }
        }
    };
    auto epilogue = [&](const W4GemmTile &t) {
        if constexpr (SWIGLU) {
            // the encoder's form (NaNs or none) by one vote a tile: 1 % of the
            // kernel against one for every four values
            bool nan = false;
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int j = 0; j < TN / 2; j++)
#pragma unroll
                    for (int v = 0; v < 16; v++) {
                        acc[j][i][v] = silu_f(acc[j][i][v]) * acc[j + TN / 2][i][v];
                        nan |= __builtin_isnan(acc[j][i][v]);
                    }
            auto finite = [](float x, float y, float z, float w, uint32_t sb) { return e4m3x4_finite(x, y, z, w, sb); };
            auto any = [](float x, float y, float z, float w, uint32_t sb) { return e4m3x4_select(x, y, z, w, sb); };
            if (__ballot(nan) == 0) store_hidden(t, finite);
            else store_hidden(t, any);
        } else {
#pragma unroll
            for (int i = 0; i < TM; i++) {
                const int row = t.row0 + wm * WTM + i * 32 + (lane & 15);
                uint16_t *c = reinterpret_cast<uint16_t *>(g.c) + (int64_t)row * N + 8 * half + (lane & 16);
                uint32_t exps = 0;                                // of the TN blocks (kOutHalf)
#pragma unroll
                for (int j = 0; j < TN; j++) {
                    const int n = t.nt * BN + wn * WTN + j * 32;
                    if (n >= N) continue;                         // wave-uniform
                    const f32x16 &f = acc[j][i];
                    float mult = 1.f;
                    if constexpr (OUT == kOutHalf) {
                        float am = 0.f;
#pragma unroll
                        for (int v = 0; v < 16; v++) am = fmaxf(am, fabsf(f[v]));
                        // the largest to 2^14 .. 2^15
                        const int sb = max((int)(__float_as_uint(max_xor32(am)) >> 23) - 14, 0);
                        mult = __uint_as_float((uint32_t)(254 - sb) << 23);
                        exps |= (uint32_t)sb << (8 * j);
                    }
                    auto pack = [&](float a, float b) {
                        if constexpr (OUT == kOutHalf) return pack_f16x2(a * mult, b * mult);
                        else return pack_bf16x2(a, b);
                    };
                    uint32_t o[2][4];
#pragma unroll
                    for (int q = 0; q < 2; q++)
#pragma unroll
                        for (int x = 0; x < 2; x++)
                            swap32(pack(f[8 * q + 2 * x], f[8 * q + 2 * x + 1]),
                                   pack(f[8 * q + 4 + 2 * x], f[8 * q + 5 + 2 * x]), o[q][x], o[q][2 + x]);
                    // then columns 8 half + 16 (lane / 16 % 2) of rows 0-15 and of rows
                    // 16-31: 64 bytes of a row an instruction, not 32 (1 to 2 %). Past
                    // the last-level cache 268 MB in bf16 left 14 % sooner, and where a
                    // combine read them behind it both together took 4 % longer.
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        const auto r = __builtin_amdgcn_permlane16_swap(o[0][x], o[1][x], false, false);
                        o[0][x] = r[0];
                        o[1][x] = r[1];
                    }
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        if (row + 16 * q >= t.row_end) continue;
                        *reinterpret_cast<uint4 *>(c + q * 16 * N + n) =
                            make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
                    }
                }
                if constexpr (OUT == kOutHalf) {
                    // N is a multiple of 128 here: all of the blocks or none
                    const int r = t.row0 + wm * WTM + i * 32 + (lane & 31), n = t.nt * BN + wn * WTN;
                    typedef typename std::conditional<TN == 4, uint32_t, uint16_t>::type Exps;
                    static_assert(TN == 4 || TN == 2, "a store of whole words");
                    if (half == 0 && r < t.row_end && n < N)
                        *reinterpret_cast<Exps *>(g.c_scale + (int64_t)r * (N / 32) + n / 32) = (Exps)exps;
                }
            }
        }
    };

    const int first = blockIdx.x >> 3;
    if (first >= rs.total) return;                                // the whole workgroup
    issue(0, std::integral_constant<int, 0>{});
    if constexpr (STAGES > 2) issue(1, std::integral_constant<int, 1>{});
    int step = 0, buf = 0, batch = 1;
    for (int pos = first; pos < rs.total; pos += workers) {
        // (of a tile of fewer steps than stages the copies are past the next one)
        const W4GemmTile cur = (ikt == 0 ? ipos - workers : ipos) == pos ? ahead : decode(pos);
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int v = 0; v < 16; v++) acc[j][i][v] = 0.f;
        // a wave whose rows all lie past the group's end only copies
        const bool mine = cur.row0 + wm * WTM < cur.row_end;
        auto next = [&](auto q) {
            // this wave's copies of the step have landed: at most those of the
            // STAGES - 2 steps behind it may be in flight (loads return in order;
            // a store or a scale copy among them makes the wait longer, not shorter)
            constexpr int Q = decltype(q)::value;
            constexpr int BEHIND = !LINES ? (STAGES - 2) * (IPA + IPB) : STAGES == 2 ? 0 : IPA + (Q & 1) * IPB;
            if (issued - step >= STAGES - 1) wait_vmem<BEHIND>();
            else wait_vmem<0>();
            lds_sync();                  // everybody's, and the stage before has been read
            issue(buf == 0 ? STAGES - 1 : buf - 1,
                  std::integral_constant<int, (Q + STAGES - 1) & 3>{});
            if constexpr (Q == 0) {
                if constexpr (BATCHED) batch ^= 1;
                if (mine) read_scales(BATCHED ? batch : buf);
            }
            if (mine) compute(buf, q);
            if (++buf == STAGES) buf = 0;
            step++;
        };
        if constexpr (BATCHED) {
            for (int kt = 0; kt < nk; kt += 4) {
                next(std::integral_constant<int, 0>{});
                next(std::integral_constant<int, 1>{});
                next(std::integral_constant<int, 2>{});
                next(std::integral_constant<int, 3>{});
            }
        } else {
            for (int kt = 0; kt < nk; kt++) next(std::integral_constant<int, 0>{});
        }
        if (mine) epilogue(cur);
    }
}

// ---------------------------------------------------------------------------
// launchers

template <int OUT, int BM, int BN, int WM, int WN, int STAGES, int OCC>
static void w4_gemm_run(const moe_w4_gemm_desc &g, hipStream_t s) {
    constexpr int per_cu = OCC * 4 / (WM * WN);
    const int grid = (num_cus() * per_cu + 7) / 8 * 8;
    if (g.K % 512 == 0)
        w4_gemm_tiles<OUT, true, BM, BN, WM, WN, STAGES, OCC><<<grid, WM * WN * 64, 0, s>>>(g);
    else
        w4_gemm_tiles<OUT, false, BM, BN, WM, WN, STAGES, OCC><<<grid, WM * WN * 64, 0, s>>>(g);
}

// The tile by the rows of a group (r, on average over the groups that can have
// any) and the number of large tiles: large ones (128 rows x 256) move the fewest
// bytes a product, medium ones (128 x 128) where the large would not fill the two
// workgroups of every compute unit, small ones (64 x 128, in three stages) where
// the weights' stream is what counts or few have a tile at all. us, up (gathered rows
// of a random routing, K = N = 2048 unless said otherwise), small / medium / large (in
// brackets the large tiles):
//   E = 128: r = 32 52 / 67 / 69, r = 48 58 / 67 / 69, r = 64 (1024) 74 / 72 / 73, r = 128 115 /
//     112 / 102, r = 512 353 / 302 / 270
//   E = 64: r = 48 27 / 33 / 37, r = 64 (512) 36 / 34 / 38, r = 96 (640) 42 / 37.5 / 41
//   E = 32: r = 40 16 / 19 / 25, r = 64 (256) 23 / 20 / 25, r = 192 (512) 41 / 35.0 / 34.7, r =
//     256 (640) 49.5 / 46.0 / 45.6, r = 288 (704) 51 / 46.7 / 45.7
//   E = 16: r = 512 (576) 45 / 40.5 / 45, r = 576 (640) 50 / 42 / 46, r = 704 (768) 70 / 50 / 48
//   E = 8: r = 32 (64) 10.9 / 13.2 / 19.4, r = 175 (116) 13.9 / 14.5 / 20.6, r = 256 (160) 18.6 /
//     17.8 / 20.8, r = 512 (288) 27 / 27 / 30, r = 960 (512) 43 / 36.5 / 35.4, r = 1024 (544)
//     44 / 41 / 45, r = 1216 (640) 60 / 43.5 / 47, r = 1280 (672) 53 / 50 / 47
//   E = 2, K = N = 8192: r = 128 (96) 35 / 43 / 61, r = 256 (160) 55 / 50 / 61, r = 512
//     (288) 87 / 89 / 89, r = 1100 (576) 159 / 144 / 149, r = 1300 (672) 188 / 173 / 152
// The large tiles pay from where they fill the compute units' places a second time
// by some: up to 640 of them the medium ones take 3 % more to 10 % less.
template <int OUT>
static void w4_gemm_pick(const moe_w4_gemm_desc &g, hipStream_t s) {
    const int64_t groups = g.rows < g.n_groups ? g.rows : g.n_groups;
    const int64_t half = g.rows / 64 + groups, m = half > 2 * groups ? half : 2 * groups;
    const int64_t tiles = m * ((g.N + 255) / 256) / 2;
    if (g.rows <= 48 * groups || tiles <= 128) w4_gemm_run<OUT, 64, 128, 2, 2, 3, 2>(g, s);
    else if (tiles <= 640) w4_gemm_run<OUT, 128, 128, 2, 2, 2, 2>(g, s);
    else w4_gemm_run<OUT, 128, 256, 2, 2, 2, 2>(g, s);
}

// MOE_EPI_NONE with a c_scale: kOutHalf
moe_status w4_gemm_launch(const moe_w4_gemm_desc &g, hipStream_t s) {
    if (g.epilogue == MOE_EPI_SWIGLU_FWD) w4_gemm_pick<kOutHidden>(g, s);
    else if (g.c_scale) w4_gemm_pick<kOutHalf>(g, s);
    else w4_gemm_pick<kOutBf16>(g, s);
    return launch_status();
}

// out[t] = sum_j g[t, j] y[token_pos[t, j]], y as kOutHalf leaves it, sums in fp32:
// a token a wave, all loads of kUnrollY column chunks in flight before the first
// sum. A lane reads one block's exponent of those chunks and hands it to the four
// that need it. Bound by memory (16384 tokens of 4 rows of
// 2048: 343 MB in 54 us, 6.4 TB/s). With five to eight rows it has 200 registers, two
// waves a SIMD: 5.4 TB/s with 5 and 6, 4.6 with 8.
constexpr int kUnrollY = 4;
template <int KMAX>
__global__ __launch_bounds__(256) void w4_combine_half(const uint4 *__restrict__ y, const uint8_t *__restrict__ scale,
                                                       const float *__restrict__ gate,
                                                       const int32_t *__restrict__ token_pos, int64_t T, int nv,
                                                       int k, uint4 *__restrict__ out) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    int32_t pos[KMAX];
    float g[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; j++) {
        pos[j] = j < k ? token_pos[t * k + j] : -1;
        g[j] = j < k ? gate[t * k + j] : 0.f;
    }
    for (int base = 0; base < nv; base += 64 * kUnrollY) {
        uint4 v[kUnrollY][KMAX];
        int e[KMAX];
#pragma unroll
        for (int j = 0; j < KMAX; j++) {
            e[j] = 0;
            if (pos[j] < 0) continue;
            const int64_t row = (int64_t)pos[j] * nv;
            if (lane < 16 * kUnrollY && base + 4 * lane < nv) e[j] = scale[(row + base) / 4 + lane];
#pragma unroll
            for (int u = 0; u < kUnrollY; u++)
                if (base + 64 * u + lane < nv) v[u][j] = load_once(y + row + base + 64 * u + lane);
        }
#pragma unroll
        for (int u = 0; u < kUnrollY; u++) {
            float acc[8] = {};
#pragma unroll
            for (int j = 0; j < KMAX; j++) {
                const int ex = __shfl(e[j], 16 * u + lane / 4) - 127;
                if (pos[j] < 0) continue;
                const uint32_t w[4] = {v[u][j].x, v[u][j].y, v[u][j].z, v[u][j].w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const f16x2 f = __builtin_bit_cast(f16x2, w[i]);
                    acc[2 * i] = fmaf(g[j], ldexpf((float)f.x, ex), acc[2 * i]);
                    acc[2 * i + 1] = fmaf(g[j], ldexpf((float)f.y, ex), acc[2 * i + 1]);
                }
            }
            const int c = base + 64 * u + lane;
            if (c < nv)
                out[t * nv + c] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                             pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
        }
    }
}

static size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// H' in MXFP8 [R, h], its scales, y fp16 [R, d], its scales
size_t w4_experts8_ws_bytes(int64_t R, int d, int h) {
    return round256((size_t)R * h) + round256((size_t)R * (h / 32)) + round256((size_t)R * d * 2) +
           round256((size_t)R * (d / 32));
}

moe_status w4_experts8_launch(const moe_w4_desc &w, const uint8_t *x_scale, hipStream_t s) {
    const int64_t R = w.T * w.k;
    uint8_t *hq = (uint8_t *)w.ws, *hs = hq + round256((size_t)R * w.h);
    uint8_t *y = hs + round256((size_t)R * (w.h / 32)), *ys = y + round256((size_t)R * w.d * 2);
    moe_w4_gemm_desc g = {};
    g.n_groups = w.E;
    g.rows = R;
    g.offsets = w.offsets;
    g.epilogue = MOE_EPI_SWIGLU_FWD;
    g.N = 2 * w.h; g.K = w.d;
    g.a = (const uint8_t *)w.x; g.a_scale = x_scale; g.a_rows = w.sorted_token;
    g.b = w.w1q; g.b_scale = w.w1_scale;
    g.c = hq; g.c_scale = hs;
    moe_status st = w4_gemm_launch(g, s);
    if (st != MOE_OK) return st;
    g.epilogue = MOE_EPI_NONE;
    g.N = w.d; g.K = w.h;
    g.a = hq; g.a_scale = hs; g.a_rows = nullptr;
    g.b = w.w2q; g.b_scale = w.w2_scale;
    g.c = y; g.c_scale = ys;
    if ((st = w4_gemm_launch(g, s)) != MOE_OK) return st;
    const int nv = w.d / 8;
    auto combine = [&](auto kmax) {
        for (int64_t t = 0; t < w.T; t += 4 * kMaxBlocks) {
            const int64_t n = w.T - t < 4 * kMaxBlocks ? w.T - t : 4 * kMaxBlocks;
            w4_combine_half<decltype(kmax)::value><<<(unsigned)((n + 3) / 4), 256, 0, s>>>(
                (const uint4 *)y, ys, w.topk_gate + t * w.k, w.token_pos + t * w.k, n, nv, w.k,
                (uint4 *)w.out + t * nv);
        }
    };
    if (w.k <= 1) combine(std::integral_constant<int, 1>{});
    else if (w.k <= 2) combine(std::integral_constant<int, 2>{});
    else if (w.k <= 4) combine(std::integral_constant<int, 4>{});
    else combine(std::integral_constant<int, 8>{});
    return launch_status();
}

}  // namespace moe
