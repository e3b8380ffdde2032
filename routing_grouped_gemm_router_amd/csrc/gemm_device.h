// gemm_device.h -- what the grouped GEMMs share on the device: the tile table
// and the XCD-aware schedule of a persistent grid, the global -> LDS copies and
// their waits, and addresses of a wave's part of an output (gemm.hip, w4_gemm.hip).
#pragma once

#include "common.h"

#define MOE_LDS __attribute__((address_space(3)))

namespace moe {

// ---------------------------------------------------------------------------
// tile table shared by the kernels

// Copies offsets[0..E] (E + 1 entries, up to 257) into LDS with a strided
// loop, so the copy is whole for any block size; ends with a barrier.
MOE_DEV void load_offsets(const int32_t *offsets, int E, int32_t *s_off) {
    for (int i = threadIdx.x; i <= E; i += blockDim.x) s_off[i] = offsets[i];
    __syncthreads();
}

// out[0] = 0, out[i + 1] = the sum of v over threads 0 .. i, for i < n with 4 <=
// n <= 256; blockDim.x >= 256. By lanes, then by waves, whose sums pass through
// out: three barriers, where a scan in LDS takes sixteen. Starts after the
// caller's last barrier and ends with one.
MOE_DEV void scan256(int32_t v, int n, int32_t *out) {
    const int tid = threadIdx.x, lane = tid & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t t = __shfl_up(v, o, 64);
        if (lane >= o) v += t;
    }
    if (tid < 256 && lane == 63) out[tid >> 6] = v;
    __syncthreads();
    const int32_t w0 = out[0], w1 = out[1], w2 = out[2];
    __syncthreads();
    if (tid < n) out[tid + 1] = v + (tid >= 64 ? w0 : 0) + (tid >= 128 ? w1 : 0) + (tid >= 192 ? w2 : 0);
    if (tid == 0) out[0] = 0;
    __syncthreads();
}

// Loads offsets[0..E] into s_off and builds s_tile[e] = sum_{e'<e} ceil(c_e'/BM).
// The scan needs blockDim.x >= 256 (E <= 256). Returns the total number of m-tiles.
MOE_DEV int build_tile_table(const int32_t *offsets, int E, int BM, int32_t *s_off,
                             int32_t *s_tile) {
    const int tid = threadIdx.x;
    load_offsets(offsets, E, s_off);
    scan256(tid < E ? (s_off[tid + 1] - s_off[tid] + BM - 1) / BM : 0, 256, s_tile);
    return s_tile[E];
}

// group of a global m-tile: largest e with s_tile[e] <= mt
MOE_DEV int find_group(const int32_t *s_tile, int E, int mt) {
    int lo = 0, hi = E;
    while (lo < hi) {
        int mid = (lo + hi + 1) >> 1;
        if (s_tile[mid] <= mt) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The same for the whole wave at once: how many of pre[1 .. n] (n <= 256, not
// decreasing) are <= v, the last i with pre[i] <= v where pre[0] is. Four reads
// in flight where the search by halves waits for eight in turn. All lanes active.
MOE_DEV int count_up_to(const int32_t *pre, int n, int v) {
    const int lane = threadIdx.x & 63;
    bool le[4];
#pragma unroll
    for (int j = 0; j < 4; j++) le[j] = 1 + lane + 64 * j <= n && pre[1 + lane + 64 * j] <= v;
    int c = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) c += __popcll(__ballot(le[j]));
    return c;
}

// silu(a) = a * sigmoid(a), the sigmoid by the hardware reciprocal (1 ulp)
// instead of a correctly rounded divide: the SwiGLU epilogues' VALU work is
// exposed between tiles (GEMM2 dgrad + SwiGLU backward 6 % faster; the
// results differ from the divided form in a few bf16 roundings)
MOE_DEV float silu_f(float a) { return a * __builtin_amdgcn_rcpf(1.f + __expf(-a)); }

// ---------------------------------------------------------------------------
// XCD-aware tile schedule
//
// MI355X has 8 XCDs with a private L2 each, and consecutive workgroup ids go
// to consecutive XCDs. The persistent grid (a multiple of 8 workgroups) is
// therefore split per XCD: workgroup b serves XCD x = b % 8 as its (b / 8)-th
// worker. Each expert's m-tiles are cut into chunks of about kChunkM m-tiles
// (below); chunk c belongs to XCD c % 8, and an XCD walks its chunks' tiles in
// order with the m-tile fastest.
// The ~32 CUs of an XCD thus work on all m-tiles of one chunk and a few of its
// weight panels at a time: each weight panel is fetched into that XCD's L2
// once and shared by all of the chunk's m-tiles, and the chunk's activation
// rows are shared by the concurrent panels. (With the n-tile fastest, the
// concurrent tiles would touch every panel of the expert and stream the whole
// weight matrix, larger than the L2, once per pair of m-tiles.)
// WGRAD gives whole experts to XCDs (hot experts are split over all XCDs, see
// build_wgrad_schedule) and orders an expert's output tiles in groups of
// kWgGroupM m-tiles, m-tile fastest within a group, so the concurrent tiles
// form a block that shares both operand panels.
// Correctness does not depend on the XCD mapping: every tile id is owned by
// exactly one workgroup.

constexpr int kMaxChunks = 1920;      // chunk list: kMaxChunks/8 entries per XCD (+1)
constexpr int kXcdChunks = kMaxChunks / 8;
#ifndef MOE_CHUNK_M
#define MOE_CHUNK_M 8
#endif
// m-tiles per chunk: an expert of fewer than twice this many stays on one XCD.
// Measured (bf16 GEMM1, GEMM2, GEMM1 dgrad): E = 8 with 32 m-tiles per expert
// 20 % faster with chunks of 8 than of 16; Zipf routing 7-8 % faster; E = 128
// (4-9 m-tiles per expert: one chunk either way) unchanged; chunks of 4 lose
// 10 % at E = 128 bf16 and MXFP8, where they split experts.
constexpr int kChunkM = MOE_CHUNK_M;
#ifndef MOE_WG_GROUP_M
#define MOE_WG_GROUP_M 8
#endif
constexpr int kWgGroupM = MOE_WG_GROUP_M;   // WGRAD: m-tiles per tile group

struct RowSchedule {
    int n_tiles;      // n-tiles per m-tile
    int chm;          // m-tiles per chunk
    int total;        // tiles owned by this workgroup's XCD
    int split;        // column parts of a chunk, as a power of two
};

// s_tile: exclusive prefix of m-tiles per group (from build_tile_table).
// Builds s_chunk (chunk prefix per group, E+1) and s_xpre (tile prefix over
// this XCD's chunks, up to kMaxChunks/8 + 1 entries). blockDim.x >= 256.
// A group of mt_e m-tiles is cut into max(1, round(mt_e / chm)) chunks of
// equal size up to one m-tile (the first mt_e % n chunks one larger): no
// chunk is a sliver that would cost its XCD a whole weight-matrix read for
// little work, and the chunks dealt to the XCDs are alike, so the XCDs'
// totals are too.
MOE_DEV int chunk_count(int mt_e, int chm) { return mt_e > 0 ? max(1, (mt_e + chm / 2) / chm) : 0; }
// m-tiles of chunk ci of a group of mt_e m-tiles, and its first m-tile
MOE_DEV int chunk_mtiles(int mt_e, int chm, int ci) {
    const int n = chunk_count(mt_e, chm);
    return mt_e / n + (ci < mt_e % n ? 1 : 0);
}
MOE_DEV int chunk_first(int mt_e, int chm, int ci) {
    const int n = chunk_count(mt_e, chm);
    return ci * (mt_e / n) + min(ci, mt_e % n);
}
// first n-tile of column part j of a chunk
MOE_DEV int part_first(int n_tiles, int split, int j) { return (n_tiles * j) >> split; }

// units > 0: the chunks are cut by columns too, into 2, 4, .. 64 equal parts, until
// there are that many of them: with few chunks some XCDs have less to do than
// others, or nothing. A weight panel is still one XCD's alone; the chunk's
// activation rows are read by several.
MOE_DEV RowSchedule build_row_schedule(const int32_t *s_tile, int E, int n_tiles, int xcd,
                                       int32_t *s_chunk, int32_t *s_xpre, int units = 0) {
    const int tid = threadIdx.x;
    const int mt_total = s_tile[E];
    // chunk size: at least kChunkM m-tiles, more when needed to stay within kMaxChunks
    const int chm = max(kChunkM, (mt_total + (kMaxChunks - 256) - 1) / (kMaxChunks - 256));
    int32_t nc = 0;
    if (tid < E) nc = chunk_count(s_tile[tid + 1] - s_tile[tid], chm);
    scan256(nc, 256, s_chunk);
    int split = 0;
    while (split < 6 && (s_chunk[E] << split) < units) split++;
    const int C = s_chunk[E] << split;
    const int cx = C > xcd ? (C - xcd + 7) / 8 : 0;     // chunks of this XCD (<= 256)
    int32_t t = 0;
    if (tid < cx) {
        const int c = xcd + 8 * tid;
        const int e = find_group(s_chunk, E, c >> split);
        const int ci = (c >> split) - s_chunk[e];
        const int mt_e = s_tile[e + 1] - s_tile[e];
        const int j = c & ((1 << split) - 1);
        t = chunk_mtiles(mt_e, chm, ci) * (part_first(n_tiles, split, j + 1) - part_first(n_tiles, split, j));
    }
    // (C <= kMaxChunks by the choice of chm, so cx <= kXcdChunks)
    scan256(t, kXcdChunks, s_xpre);
    RowSchedule r;
    r.n_tiles = n_tiles;
    r.chm = chm;
    r.split = split;
    r.total = s_xpre[cx];
    (void)cx;
    return r;
}

// position p of this XCD's list -> (group e, m-tile index within e, n-tile)
MOE_DEV void decode_row_tile(const RowSchedule &rs, const int32_t *s_tile, const int32_t *s_chunk,
                             const int32_t *s_xpre, int E, int xcd, int p, int &e, int &mt_e,
                             int &nt) {
    // the last lc with s_xpre[lc] <= p (entries past this XCD's chunk count
    // repeat the total, which is > p), then the chunk's group
    const int lc = count_up_to(s_xpre, kXcdChunks, p);
    const int u = xcd + 8 * lc, c = u >> rs.split;
    const int o = p - s_xpre[lc];
    e = count_up_to(s_chunk, E, c);
    // m-tile fastest within the chunk: the XCD's concurrent tiles cover all
    // of the chunk's m-tiles and a few weight panels, so each weight panel
    // is fetched into the XCD's L2 once and shared by the chunk's m-tiles
    const int ci = c - s_chunk[e];
    const int cm = chunk_mtiles(s_tile[e + 1] - s_tile[e], rs.chm, ci);
    mt_e = chunk_first(s_tile[e + 1] - s_tile[e], rs.chm, ci) + o % cm;
    nt = part_first(rs.n_tiles, rs.split, u & ((1 << rs.split) - 1)) + o / cm;
}

// A condition that holds for the whole wave or for none of its lanes, taken
// from lane 0 so that the branch on it is a scalar one.
MOE_DEV bool wave_full(bool c) { return __builtin_amdgcn_readfirstlane((int)c) != 0; }

// Byte address of element (row, col) of a row-major matrix with ld elements
// per row, for wave-uniform row and col (kept in scalar registers), and the
// byte offset of lane l's first accumulator element from there: row
// (l / 32) * 4, column l % 32 of the MFMA output layout.
template <typename T>
MOE_DEV char *wave_base(T *p, int row, int col, int ld) {
    row = __builtin_amdgcn_readfirstlane(row);
    col = __builtin_amdgcn_readfirstlane(col);
    return reinterpret_cast<char *>(p + ((int64_t)row * ld + col));
}
template <int ES>
MOE_DEV uint32_t lane_off(int lane, int ld) { return (uint32_t)(((lane >> 5) * 4 * ld + (lane & 31)) * ES); }

// Wait until at most N vector-memory instructions of this wave are in flight
// (they complete in issue order).
template <int N>
MOE_DEV void wait_vmem() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Workgroup barrier for the LDS pipeline: this wave's LDS reads have
// completed (lgkmcnt(0)), then s_barrier, then an acquire fence on LDS only so
// later LDS reads stay below the barrier. No global-memory fence: that would
// drain the LDS copies that are still in flight for later stages.
MOE_DEV void lds_sync() {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Copy 16 (dma16) or 4 (dma4) bytes per lane from global memory straight into
// LDS: lane l's bytes land at lds_wave_base + size * l (lds_wave_base is
// wave-uniform, passed in M0). Issued through inline asm so that the only
// waits on these copies are the explicit ones of the pipeline below
// (wait_vmem + lds_sync); the instructions have no result registers, and the
// "memory" clobber keeps LDS reads from moving across them.
MOE_DEV void dma16(const void *src, const void *lds_wave_base) {
    // wave-uniform by construction; readfirstlane keeps it in an SGPR for M0
    const uint32_t m0v = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(const MOE_LDS void *)lds_wave_base);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(src), "s"(m0v)
                 : "memory", "m0");
}
MOE_DEV void dma4(const void *src, const void *lds_wave_base) {
    // wave-uniform by construction; readfirstlane keeps it in an SGPR for M0
    const uint32_t m0v = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(const MOE_LDS void *)lds_wave_base);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
                 :
                 : "v"(src), "s"(m0v)
                 : "memory", "m0");
}

// The same copy with the address split into a wave-uniform base in SGPRs
// and a 32-bit per-lane offset: advancing a whole tile by one K step is then
// a scalar add, with no per-lane address arithmetic.
MOE_DEV void dma16s(uint32_t voff, const char *sbase, const void *lds_wave_base) {
    const uint32_t m0v = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(const MOE_LDS void *)lds_wave_base);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(voff), "s"(sbase), "s"(m0v)
                 : "memory", "m0");
}

// a pointer that is equal in every lane, moved into scalar registers (the
// builtin returns a signed int: each half is widened from uint32_t, or a low
// word with bit 31 set would be sign-extended over the high word)
MOE_DEV const char *uniform_ptr(const char *p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const char *>((uintptr_t)((hi << 32) | lo));
}

}  // namespace moe
