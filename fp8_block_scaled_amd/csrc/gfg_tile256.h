// Pieces shared by the kernels on 256 x 256 output tiles: the work tile, the
// LDS layout of a stage and a lane's fragment offsets in it (gfx950).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg_device.h"

namespace gfg {
namespace {

constexpr int BM = 256, BN = 256, BK = 128;
constexpr int NTHREADS = 256, WAVES = 4;
constexpr int A_BYTES = BM * BK;                 // 32 KB of A per stage
constexpr int STAGE = A_BYTES + BN * BK;         // + 32 KB of B
constexpr int A_DMA = A_BYTES / 1024 / WAVES;    // 1 KB DMA instructions per wave and stage
constexpr int B_DMA = BN * BK / 1024 / WAVES;
constexpr int CAND_MAX = 4096;                   // candidate M tiles (128-row contiguous, 256-row masked)
constexpr int CPT = CAND_MAX / NTHREADS;         // candidates per thread in the list build

// One work tile: contiguous: first 128-row candidate | (128 rows only) << 12 | expert << 16;
// masked: candidate (group * tiles per group + 256-row index) | valid rows << 12.
struct TileInfo {
    int g;
    int row0;   // first row of the tile inside its region (the group, for the masked layout)
    int lim;    // rows of the tile that may be read and written
    int n0;     // first output column
};

template <bool MASKED>
__device__ __forceinline__ TileInfo tile_info(const Params& p, uint32_t e, int nt) {
    TileInfo t;
    const int c = int(e & 0xFFFu);
    if (MASKED) {
        t.g = c / p.mt_per_group;
        t.row0 = (c - t.g * p.mt_per_group) * BM;
        t.lim = int(e >> 12);
    } else {
        t.g = int(e >> 16);
        t.row0 = c * 128;
        t.lim = min(((e >> 12) & 1u) ? 128 : BM, int(p.rows) - t.row0);
    }
    t.n0 = nt * BN;
    t.g = __builtin_amdgcn_readfirstlane(t.g);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.lim = __builtin_amdgcn_readfirstlane(t.lim);
    t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
    return t;
}

// Block-wide exclusive scan (sum, or max with identity -1) over the NTHREADS threads.
template <bool MAX>
__device__ __forceinline__ int block_exclusive_scan(int v, GFG_LDS int* tmp, int lane, int wave, int* total) {
    int x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d, 64);
        if (lane >= d) x = MAX ? max(x, y) : x + y;
    }
    if (lane == 63) tmp[wave] = x;
    __syncthreads();
    int pre = MAX ? -1 : 0, all = MAX ? -1 : 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const int tw = tmp[w];
        if (w < wave) pre = MAX ? max(pre, tw) : pre + tw;
        all = MAX ? max(all, tw) : all + tw;
    }
    int ex = __shfl_up(x, 1, 64);
    if (lane == 0) ex = MAX ? -1 : 0;
    __syncthreads();   // tmp is reused by the next scan
    *total = all;
    return MAX ? max(pre, ex) : pre + ex;
}

// LDS layout of a stage: 128-byte rows, A (256 rows) then B (256 rows), both
// as the 128-row kernel's A tile: LDS row R holds tile row a_row(R) =
// R ^ ((R >> 2) & 1) and its physical 16-byte chunk c the logical chunk
// c ^ ((R >> 2) & 7).  A 16x16x128 fragment takes rows 4 apart (row
// 64 h + 4 l16 + f of the wave's 128), so a lane's four rows share one
// A-scale dword, and the row-parity exchange keeps the fragment reads free of
// bank conflicts.  DMA chunk j of wave w fills LDS rows 8 (4 j + w) .. +7;
// with four waves chunk j is chunk 0 moved by 32 j rows (a_row and the chunk
// key do not depend on j).
__device__ __forceinline__ int a_row(int p) { return p ^ ((p >> 2) & 1); }   // an involution
__device__ __forceinline__ int swz_a(int p, int c) { return p * BK + ((c ^ ((p >> 2) & 7)) << 4); }

struct LaneOffsets {
    uint32_t a0;   // A chunk 0; chunk j adds 32 j rows
    uint32_t b0;   // B chunk 0; chunk j adds 32 j rows
    uint32_t K;    // row stride (uniform)
};

// The lane index, read afresh where it is used: values derived from it ahead
// of the tile loop would stay live (and be spilled) through the K loop.
__device__ __forceinline__ int lane_now() {
    int ln;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(ln));
    return ln;
}

// The lane's DMA source offset of chunk 0 (A and B alike), from the lane index
// read afresh: computed per step, it is not held through the step's first half.
// Chunk 0 of wave w covers LDS rows R = 8 w + (lane >> 3); lane i writes
// physical chunk i % 8, the logical chunk (i % 8) ^ ((R >> 2) & 7) of tile row
// a_row(R).
__device__ __forceinline__ uint32_t dma_lane_offset(int wave, uint32_t K) {
    const int ln = lane_now();
    const int R = 8 * wave + (ln >> 3);
    return uint32_t(a_row(R)) * K + uint32_t(((ln & 7) ^ ((R >> 2) & 7)) << 4);
}

struct Lane {
    // LDS offsets of this lane's fragment rows for the first 64-row half and
    // fragment f = 0 (row p0 + odd for even f, p0 - odd for odd f, then + f
    // rows); logical chunks lq (lo) and lq + 4 (hi).  The second half adds 64
    // rows.  B offsets include the A region.
    int a_lo_e, a_lo_o, a_hi_e, a_hi_o;
    int b_lo_e, b_lo_o, b_hi_e, b_hi_o;
    LaneOffsets off;     // DMA source offsets
    int wave, wm, wn, sa_off;
};

__device__ __forceinline__ int frag_off(int e, int o, int y) {
    const int f = y & 3;
    return ((f & 1) ? o : e) + f * BK + (y >> 2) * 64 * BK;
}

#define GFG_SB() __builtin_amdgcn_sched_barrier(0)


__device__ __forceinline__ u32x4 lds16(const GFG_LDS uint8_t* __restrict__ src, int a) {
    return *reinterpret_cast<const GFG_LDS u32x4*>(src + a);
}
// The row mask of a lane: bit y set when its output row for fragment y may be
// written (inside the tile's rows and, for the contiguous layout, of the
// tile's expert).
template <bool MASKED>
__device__ __forceinline__ int row_mask(const Lane& L, const u32x4 (&lay)[2], int lim, int g) {
    int okm = 0;
#pragma unroll
    for (int y = 0; y < 8; ++y)
        okm |= int(L.sa_off + 64 * (y >> 2) + (y & 3) < lim && (MASKED || int(lay[y >> 2][y & 3]) == g)) << y;
    return okm;
}

}  // namespace
}  // namespace gfg
