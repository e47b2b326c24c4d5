// 8-bit integer matrix product on 256 x 256 or 192 x 256 output tiles for gfx950
// (MI355X): the launches that 128 x 128 tiles would take in several rounds.
//
//   d[m, n] = (sum_k a[m, k] b[n, k]) * a_scale[m] * b_scale[n] (+ bias[n])
//
// Design: four wave64s, one per SIMD, each owning a 128 x 128 quarter of the
// tile: 256 accumulator registers (64 16x16 blocks of 32-bit sums) and 192
// fragment registers.  K goes in steps of 128 bytes through two 64 KB LDS
// stages filled by direct-to-LDS loads; a 16 x 16 block takes two
// v_mfma_i32_16x16x64_i8 a step, one for the chunks 0..3 of its rows' 128
// bytes and one for the chunks 4..7 (K's order inside a step is the same for
// both operands, and the sums are exact, so it is free).  The two MFMAs of a
// block are kept apart by its neighbour's, since the second adds to the first.
// Alone on its SIMD, a wave's instruction order is the schedule, so every
// group of instructions is pinned in place: a step has two barriers, the first
// frees the rows of the stage whose fragments are already in registers, whose
// refill then runs under the step's own MFMAs, the second waits for the next
// stage.  The refills of a tile's last two steps load the next tile's first
// two stages.
//
// What bounds it: with every CU busy, a wave alone on its SIMD, whose own loads,
// LDS reads and barriers hold up its MFMAs, at the clock that the chip holds under
// this load; between tiles, the epilogue.  8 x 4096 x 7168 at five depths fits 1.58
// us a step and 6.2 us a tile (the FP8 kernel beside it: 1.53 and 3.2); a tile
// alone on the chip takes 1.05 us a step, 0.90 with 192 rows.  Counters: 4096 x 4096 x
// 16384, 199-219 us, 2510-2760 TOP/s (a library's product: 2408): the matrix pipes are
// busy 67% of the time at 1.97 GHz, each CU takes in 42 GB/s from L2, no LDS bank
// conflicts; 8 x 4096 x 7168 x 2304, 470-496 us, 2180-2300: 51% at 2.06 GHz, 34 GB/s; the
// masked 8 x up to 1024 rows x 2048 x 7168, one round of 192-row tiles, 87-90 us: 37%
// at 2.4 GHz, 32 GB/s.
//
// Rows of a tile: 192 where 7/8 of its rounds over the CUs beat the 256-row
// tile's (a 192-row tile moves 7/8 of the bytes).  Measured, us, 192 and 256:
// 2000 x 4096 x 4096 (176, 128 tiles) 39.9, 45.1; 768 x 7168 x 2304 (112, 84)
// 26.3, 30.0; 5000 x 7168 x 2304 (756, 560: three rounds either way) 82.8, 91.1; but
// 8192 x 7168 x 2304 (1204, 896: 5 and 4) 138.8, 130.1; 4096 x 4096 x 16384 (352,
// 256: 2 and 1) 281, 205.  (The contiguous layout's experts start at 128-row
// tiles, which 192 does not divide: 256 there.)
//
// Sizes that are no multiple of the tile cost nothing inside the loop: rows
// past an operand's end and chunks past K have load offsets outside the buffer
// window, where the hardware returns zeros, and K is rounded up to an even
// number of steps.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_int8.h"
#include "gfg_internal.h"
#include "gfg_tile256.h"

namespace gfg {
namespace {

constexpr uint32_t kOutside = 0x80000000u;       // past every buffer window used here (all below 2^31 bytes)
constexpr int FIRST_HALF = 12;                   // a step's loads issued before its mid barrier (of 16)

// The work tiles of TM rows in M order, in `work`; returns their number.  Uses
// the stage buffer `buf0` (before the first DMA) for the candidates' experts.
template <bool MASKED, int TM>
__device__ __forceinline__ int build_work_list(const I8Params& p, GFG_LDS uint8_t* buf0, uint32_t* work, int tid, int lane,
                                               int wave) {
    GFG_LDS int* const expo = reinterpret_cast<GFG_LDS int*>(buf0);   // [CAND_MAX]
    GFG_LDS int* const tmp = expo + CAND_MAX;
    const int per = int((p.rows + TM - 1) / TM), n_cand = MASKED ? p.G * per : p.m_tiles;
    const int c0 = tid * CPT;     // this thread's CPT consecutive candidates
    unsigned wmask = 0;           // bit j: candidate c0 + j starts a work tile
    unsigned hmask = 0;           // contiguous: ... that has only 128 rows (its run ends with it)
    if (MASKED) {
        // candidate g * per + j: rows [TM j, TM j + TM) of group g
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = c0 + j;
            if (c < n_cand) {
                const int g = c / per;
                int mm = p.meta[g];
                mm = mm < 0 ? 0 : (mm > p.rows ? int(p.rows) : mm);
                if (mm - (c - g * per) * TM > 0) wmask |= 1u << j;
            }
        }
    } else {
        // candidate c: the 128-row tile starting at row 128 c; its expert is
        // that of its first row.  A run is a maximal stretch of candidates of
        // one expert; work tiles start at even offsets inside a run.
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = c0 + j;
            if (c < p.m_tiles) {
                const int e = p.meta[int64_t(c) * 128];
                expo[c] = e >= 0 && e < p.G ? e : -1;
            }
        }
        __syncthreads();
        int last_start = -1;
        int e_prev = (c0 > 0 && c0 - 1 < p.m_tiles) ? expo[c0 - 1] : -1;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = c0 + j;
            if (c < p.m_tiles) {
                const int e = expo[c];
                if (e >= 0 && e != e_prev) last_start = c;
                e_prev = e;
            }
        }
        int unused;
        int run_start = block_exclusive_scan<true>(last_start, tmp, lane, wave, &unused);
        e_prev = (c0 > 0 && c0 - 1 < p.m_tiles) ? expo[c0 - 1] : -1;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = c0 + j;
            if (c < p.m_tiles) {
                const int e = expo[c];
                if (e >= 0 && e != e_prev) run_start = c;
                e_prev = e;
                if (e >= 0 && ((c - run_start) & 1) == 0) {
                    wmask |= 1u << j;
                    if (!(c + 1 < p.m_tiles && expo[c + 1] == e)) hmask |= 1u << j;
                }
            }
        }
    }
    int n_work;
    int off = block_exclusive_scan<false>(__popc(wmask), tmp, lane, wave, &n_work);
#pragma unroll
    for (int j = 0; j < CPT; ++j)
        if ((wmask >> j) & 1u) {
            const int c = c0 + j;
            uint32_t e;
            if (MASKED) {
                const int g = c / per;
                int mm = p.meta[g];
                mm = mm < 0 ? 0 : (mm > p.rows ? int(p.rows) : mm);
                e = uint32_t(c) | (uint32_t(min(mm - (c - g * per) * TM, TM)) << 12);
            } else {
                e = uint32_t(c) | (((hmask >> j) & 1u) << 12) | (uint32_t(expo[c]) << 16);
            }
            work[off++] = e;
        }
    return n_work;
}

// What the refills of one tile read: its A rows and its B rows.
struct Source {
    __amdgpu_buffer_rsrc_t a, b;
};

template <int LAYOUT, int TM>
__device__ __forceinline__ TileInfo tile_of(const I8Params& p, const uint32_t* work, int mr, int nt) {
    TileInfo t;
    if (LAYOUT == DENSE) {
        t.g = 0;
        t.row0 = mr * TM;
        t.lim = int(p.rows - t.row0 < TM ? p.rows - t.row0 : TM);
    } else {
        const uint32_t e = work[mr];
        const int c = int(e & 0xFFFu);
        if (LAYOUT == MASKED) {
            const int per = int((p.rows + TM - 1) / TM);
            t.g = c / per;
            t.row0 = (c - t.g * per) * TM;
            t.lim = int(e >> 12);
        } else {
            t.g = int(e >> 16);
            t.row0 = c * 128;
            t.lim = min(((e >> 12) & 1u) ? 128 : BM, int(p.rows) - t.row0);
        }
    }
    t.n0 = nt * BN;
    t.g = __builtin_amdgcn_readfirstlane(t.g);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.lim = __builtin_amdgcn_readfirstlane(t.lim);
    t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
    return t;
}

template <int LAYOUT>
__device__ __forceinline__ Source source_of(const I8Params& p, const TileInfo& t) {
    const int64_t region = LAYOUT == MASKED ? int64_t(t.g) * p.rows : 0;
    const int cols = min(BN, p.N - t.n0);
    return Source{make_rsrc(p.a + (region + t.row0) * p.K, uint32_t(t.lim) * uint32_t(p.K)),
                  make_rsrc(p.b + (int64_t(t.g) * p.N + t.n0) * p.K, uint32_t(cols) * uint32_t(p.K))};
}

// The lane's source offset of chunk 0 of stage kb (A and B alike): row
// a_row(R) of the tile, R = 8 wave + (lane >> 3), 16-byte chunk (lane & 7) ^
// ((R >> 2) & 7) of the step; outside the window when that chunk lies past K.
__device__ __forceinline__ uint32_t stage_offset(int wave, int kb, int K) {
    const int ln = lane_now();
    const int R = 8 * wave + (ln >> 3);
    const int k = kb * BK + (((ln & 7) ^ ((R >> 2) & 7)) << 4);
    return k < K ? uint32_t(a_row(R)) * uint32_t(K) + uint32_t(k) : kOutside;
}

// The same for A's chunks of two-row fragments (below).
__device__ __forceinline__ uint32_t stage_offset2(int wave, int kb, int K) {
    const int ln = lane_now();
    const int R = 8 * wave + (ln >> 3);
    const int k = kb * BK + (((ln & 7) ^ ((R >> 1) & 7)) << 4);
    return k < K ? uint32_t(R ^ ((R >> 1) & 1)) * uint32_t(K) + uint32_t(k) : kOutside;
}

// Load chunk c (0..7: A's, 8..15: B's) of a stage: 32 (c & 7) rows further on.
__device__ __forceinline__ void refill(const Source& r, uint32_t off, int K, GFG_LDS uint8_t* dst, int wave, int c) {
    asm volatile("" : "+v"(off));   // added per chunk, not eight offsets held live
    const int j = c & 7;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(c < 8 ? r.a : r.b, (GFG_LDS void*)(dst + (j * WAVES + wave) * 1024), 16,
                                             off + uint32_t(32 * j) * uint32_t(K), 0, 0, 0);
}

__device__ __forceinline__ v4i lds_frag(const GFG_LDS uint8_t* __restrict__ src, int a) {
    return *reinterpret_cast<const GFG_LDS v4i*>(src + a);
}

// 16 and 4 bytes at any column
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t uint32_at2 __attribute__((aligned(2)));

struct Frag { v4i lo, hi; };

__device__ __forceinline__ v4i mma(const v4i& b, const v4i& a, const v4i& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0);
}

// Tiles of 256 or 192 rows: a wave has MY = 8 or 6 fragment rows of A.  Those
// of 256: fragments y of two 64-row halves, rows 64 (y >> 2) + 4 l16 + (y & 3).
// Those of 192: four fragments of 64 rows, as before, and two of the other 32,
// rows 64 + 2 l16 + (y - 4); the LDS rows of these are exchanged and swizzled
// by bit 1 and bits 1..3 of the row in place of bit 2 and bits 2..4, so that a
// fragment's lanes read the same banks as before.  32 rows are a chunk of
// loads, so a chunk is of one kind.
struct LaneA2 { int lo_e, lo_o, hi_e, hi_o; };      // LDS offsets of fragments 4 and 5 of 6

template <int MY>
__device__ __forceinline__ int a_off(const Lane& L, const LaneA2& L2, int y, bool hi) {
    if (MY == 8 || y < 4) return hi ? frag_off(L.a_hi_e, L.a_hi_o, y) : frag_off(L.a_lo_e, L.a_lo_o, y);
    return y == 4 ? (hi ? L2.hi_e : L2.lo_e) : (hi ? L2.hi_o : L2.lo_o) + BK;
}

// One step k: stage k in `cur` (its B region also as `cur_b`), stage k+1 in
// `nxt`; stage kr refills `cur`.  On entry af[0..3] and bc hold stage k's A
// fragments 0..3 and B fragments.  First half: MY / 2 fragment rows, whose
// first slots read A's other fragments, with 12 refills of the rows already
// read; second half: the other fragment rows, the last refills, and stage
// k+1's B fragments and A fragments 0..3 (of 6, fragment 3 is still in use in
// the first eight slots).  VMWAIT: vector-memory operations issued after stage
// k+1's last load that may still be in flight at the mid barrier.
template <int VMWAIT, int MY>
__device__ __forceinline__ void i8_step(const Lane& L, const LaneA2& L2, int K, GFG_LDS uint8_t* __restrict__ cur,
                                        GFG_LDS uint8_t* __restrict__ cur_b, GFG_LDS uint8_t* __restrict__ nxt, int kr,
                                        const Source& rf, v4i (&acc)[MY][8], Frag (&af)[MY], Frag (&bc)[8], Frag (&bn)[8]) {
    constexpr int HALF = MY / 2, LATE = 2 * (MY - 4), EVERY = MY == 8 ? 2 : 1;
    GFG_SB();
    GFG_WAITCNT(63, 0);
    __builtin_amdgcn_s_barrier();
    GFG_SB();
    const uint32_t off = stage_offset(L.wave, kr, K);
    const uint32_t off2 = MY == 8 ? off : stage_offset2(L.wave, kr, K);
    GFG_SB();
#pragma unroll
    for (int m = 0; m < 8 * HALF; ++m) {
        const int y = m >> 3, x = m & 6;
        if (!(m & 1)) {
            acc[y][x] = mma(bc[x].lo, af[y].lo, acc[y][x]);
            acc[y][x + 1] = mma(bc[x + 1].lo, af[y].lo, acc[y][x + 1]);
        } else {
            acc[y][x] = mma(bc[x].hi, af[y].hi, acc[y][x]);
            acc[y][x + 1] = mma(bc[x + 1].hi, af[y].hi, acc[y][x + 1]);
        }
        GFG_SB();
        if (m < LATE) {
            const int yy = 4 + (m >> 1);
            if (m & 1) af[yy].hi = lds_frag(cur, a_off<MY>(L, L2, yy, true));
            else af[yy].lo = lds_frag(cur, a_off<MY>(L, L2, yy, false));
            GFG_SB();
        }
        if (m >= LATE && m < LATE + 12 * EVERY && m % EVERY == 0) {
            const int q = (m - LATE) / EVERY;        // A's chunks of fragments 0..3 (0, 1 and 4, 5, or 3, 4), then B's
            if (q < 4) refill(rf, off, K, cur, L.wave, (q & 1) + HALF * (q >> 1));
            else refill(rf, off, K, cur_b, L.wave, 8 + q - 4);
            GFG_SB();
        }
    }
    GFG_WAITCNT(VMWAIT, 0);
    __builtin_amdgcn_s_barrier();
    GFG_SB();
#pragma unroll
    for (int m = 0; m < 8 * (MY - HALF); ++m) {
        const int y = HALF + (m >> 3), x = m & 6;
        if (!(m & 1)) {
            acc[y][x] = mma(bc[x].lo, af[y].lo, acc[y][x]);
            acc[y][x + 1] = mma(bc[x + 1].lo, af[y].lo, acc[y][x + 1]);
        } else {
            acc[y][x] = mma(bc[x].hi, af[y].hi, acc[y][x]);
            acc[y][x + 1] = mma(bc[x + 1].hi, af[y].hi, acc[y][x + 1]);
        }
        GFG_SB();
        if (MY == 8 && (m & 7) == 1) refill(rf, off, K, cur, L.wave, 2 + ((m >> 3) & 1) + 4 * (m >> 4));   // chunks 2, 3, 6, 7
        if (MY == 6 && (m & 7) == 1 && m < 16) refill(rf, off2, K, cur, L.wave, 2 + 3 * (m >> 3));         // chunks 2, 5
        if (m < 16) {
            const int xx = m >> 1;
            if (m & 1) bn[xx].hi = lds_frag(nxt, frag_off(L.b_hi_e, L.b_hi_o, xx));
            else bn[xx].lo = lds_frag(nxt, frag_off(L.b_lo_e, L.b_lo_o, xx));
        } else if (m < 24) {
            const int yy = (m - 16) >> 1;
            if (m & 1) af[yy].hi = lds_frag(nxt, a_off<MY>(L, L2, yy, true));
            else af[yy].lo = lds_frag(nxt, a_off<MY>(L, L2, yy, false));
        }
        GFG_SB();
    }
}

// The launch's tiles of 32 MY rows.
template <int LAYOUT, int MY, typename OutT>
__device__ __forceinline__ void walk_tiles(const I8Params& p, GFG_LDS uint8_t* buf0, GFG_LDS uint8_t* buf1, uint32_t* work, int tid,
                                           int lane, int wave) {
    constexpr int TM = 32 * MY;
    int n_work = int((p.rows + TM - 1) / TM);
    if (LAYOUT != DENSE) {
        n_work = build_work_list<LAYOUT == MASKED, TM>(p, buf0, work, tid, lane, wave);
        n_work = __builtin_amdgcn_readfirstlane(n_work);
        __syncthreads();   // the list is complete, and stage buffer 0 is free for the loads
    }
    const int NT = (p.N + BN - 1) / BN;
    TileOrder order;
    order.init(unsigned(n_work) * unsigned(NT), p.num_xcd);
    order.x_start = __builtin_amdgcn_readfirstlane(order.x_start);
    order.x_count = __builtin_amdgcn_readfirstlane(order.x_count);
    order.slot = __builtin_amdgcn_readfirstlane(order.slot);
    order.slots = __builtin_amdgcn_readfirstlane(order.slots);
    const unsigned gm = p.group_m > 0 ? unsigned(p.group_m) : 4u;
    unsigned i = order.slot;
    if (i >= order.x_count) return;

    Lane L;
    LaneA2 L2{};
    L.wave = wave;
    L.wm = wave >> 1;
    L.wn = wave & 1;
    const int l16 = lane & 15, lq = lane >> 4, odd16 = l16 & 1;
    {
        const int p0 = L.wm * (16 * MY) + 4 * l16, pb = L.wn * 128 + 4 * l16;
        L.a_lo_e = swz_a(p0, lq) + odd16 * BK;
        L.a_lo_o = swz_a(p0, lq) - odd16 * BK;
        L.a_hi_e = swz_a(p0, lq + 4) + odd16 * BK;
        L.a_hi_o = swz_a(p0, lq + 4) - odd16 * BK;
        if (MY == 6) {
            const int p2 = (L.wm * 96 + 64 + 2 * l16) * BK, lo = (lq ^ (l16 & 7)) << 4, hi = ((lq + 4) ^ (l16 & 7)) << 4;
            L2 = LaneA2{p2 + lo + odd16 * BK, p2 + lo - odd16 * BK, p2 + hi + odd16 * BK, p2 + hi - odd16 * BK};
        }
        L.b_lo_e = A_BYTES + swz_a(pb, lq) + odd16 * BK;
        L.b_lo_o = A_BYTES + swz_a(pb, lq) - odd16 * BK;
        L.b_hi_e = A_BYTES + swz_a(pb, lq + 4) + odd16 * BK;
        L.b_hi_o = A_BYTES + swz_a(pb, lq + 4) - odd16 * BK;
    }
    const int KB = ((p.K + BK - 1) / BK + 1) & ~1;   // an even number of steps; those past K add zeros
    __builtin_assume(KB >= 2);
    int mr, nt;
    order.item(i, gm, unsigned(NT), unsigned(n_work), &mr, &nt);
    TileInfo cur = tile_of<LAYOUT, TM>(p, work, mr, nt);
    Source rf = source_of<LAYOUT>(p, cur);

    v4i acc[MY][8];
    Frag af[MY], bf0[8], bf1[8];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint32_t off = stage_offset(wave, s, p.K), off2 = MY == 8 ? off : stage_offset2(wave, s, p.K);
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < MY || c >= 8)
                refill(rf, MY == 6 && (c == 2 || c == 5) ? off2 : off, p.K, (s ? buf1 : buf0) + (c < 8 ? 0 : A_BYTES), wave, c);
    }
    GFG_WAITCNT(0, 15);
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int y = 0; y < 4; ++y)
        af[y] = Frag{lds_frag(buf0, a_off<MY>(L, L2, y, false)), lds_frag(buf0, a_off<MY>(L, L2, y, true))};
#pragma unroll
    for (int x = 0; x < 8; ++x)
        bf0[x] = Frag{lds_frag(buf0, frag_off(L.b_lo_e, L.b_lo_o, x)), lds_frag(buf0, frag_off(L.b_hi_e, L.b_hi_o, x))};

    while (true) {
#pragma unroll
        for (int y = 0; y < MY; ++y)
#pragma unroll
            for (int x = 0; x < 8; ++x) acc[y][x] = v4i{};
        i = __builtin_amdgcn_readfirstlane(i);
        const unsigned i_next = i + order.slots;
        const bool have_next = i_next < order.x_count;
        TileInfo next = cur;
        if (have_next) {
            int mr2, nt2;
            order.item(i_next, gm, unsigned(NT), unsigned(n_work), &mr2, &nt2);
            next = tile_of<LAYOUT, TM>(p, work, mr2, nt2);
        }
        // Step k refills with stage k + 2; from step KB - 2 on with the next
        // tile's stage k + 2 - KB, or, on the last tile, with nothing (a stage
        // past K lies outside the window).
        auto stage_of = [&](int k) { return k + 2 < KB ? k + 2 : (have_next ? k + 2 - KB : KB); };
        // The first pair: stage 1 has landed already (everything before the
        // previous tile's scale loads, or before the first tile, has).
        if (KB == 2 && have_next) rf = source_of<LAYOUT>(p, next);
        i8_step<63, MY>(L, L2, p.K, buf0, buf0 + A_BYTES, buf1, stage_of(0), rf, acc, af, bf0, bf1);
        i8_step<FIRST_HALF, MY>(L, L2, p.K, buf1, buf1 + A_BYTES, buf0, stage_of(1), rf, acc, af, bf1, bf0);
        for (int kb = 2; kb < KB; kb += 2) {
            if (kb + 2 == KB && have_next) rf = source_of<LAYOUT>(p, next);
            i8_step<FIRST_HALF, MY>(L, L2, p.K, buf0, buf0 + A_BYTES, buf1, stage_of(kb), rf, acc, af, bf0, bf1);
            i8_step<FIRST_HALF, MY>(L, L2, p.K, buf1, buf1 + A_BYTES, buf0, stage_of(kb + 1), rf, acc, af, bf1, bf0);
        }

        // ---- epilogue.  Lane (l16, lq) holds, for each y, the output row of
        // A's fragment row (row_of), and for each column half hx
        // columns 128 wn + 64 hx + 16 lq + 4 i + x in acc[y][4 hx + x][i].
        const int ln = lane_now();
        const int64_t out_row0 = (LAYOUT == MASKED ? int64_t(cur.g) * p.rows : 0) + cur.row0;
        const int cols = min(BN, p.N - cur.n0);
        const int c0 = L.wn * 128 + 16 * (ln >> 4);
        const auto sar = make_rsrc(p.a_scale + out_row0, uint32_t(cur.lim) * 4u);
        const auto sbr = make_rsrc(p.b_scale + int64_t(cur.g) * p.N + cur.n0, uint32_t(cols) * 4u);
        const auto bir = make_rsrc(p.bias ? p.bias + cur.n0 : p.b_scale, p.bias ? uint32_t(cols) * 4u : 0u);
        const auto lar = make_rsrc(LAYOUT == CONTIG ? p.meta + cur.row0 : (const int32_t*)p.b_scale,
                                   LAYOUT == CONTIG ? uint32_t(cur.lim) * 4u : 0u);
        auto row_of = [&](int l16, int y) {
            if (MY == 8) return L.wm * 128 + 64 * (y >> 2) + 4 * l16 + (y & 3);
            return L.wm * 96 + (y < 4 ? 4 * l16 + y : 64 + 2 * l16 + y - 4);
        };
        float sa[MY];
        int okm = 0;
#pragma unroll
        for (int y = 0; y < MY; ++y) {
            const int r = row_of(ln & 15, y);
            sa[y] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sar, uint32_t(r) * 4u, 0, 0));
            bool ok = r < cur.lim;
            if (LAYOUT == CONTIG) ok = ok && int(__builtin_amdgcn_raw_buffer_load_b32(lar, uint32_t(r) * 4u, 0, 0)) == cur.g;
            okm |= int(ok) << y;
        }
        // rows of an even number of columns start at dwords, where the buffer
        // stores can write; cut: the tile ends inside a chunk of eight columns
        const bool dwords = (p.N & 1) == 0, cut = (cols & 7) != 0;
        uint8_t* const out = reinterpret_cast<uint8_t*>(p.d) + (out_row0 * p.N + cur.n0) * 2;
        const __amdgpu_buffer_rsrc_t dr = make_rsrc(out,
                                                    uint32_t(cur.lim) * uint32_t(p.N) * 2u);
        // per slot h, the row bits of the pair lane whose rows the slot holds after the exchange
        const int okh[2] = {__builtin_amdgcn_update_dpp(0, okm, 0xA0, 0xF, 0xF, false),
                            __builtin_amdgcn_update_dpp(0, okm, 0xF5, 0xF, 0xF, false)};
        const bool odd = (ln & 1) != 0;
#pragma unroll
        for (int hx = 0; hx < 2; ++hx) {
            // scale and bias of column c0 + 64 hx + 4 i + x in [i][x]
            float sb[4][4], bi[4][4];
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t co = uint32_t(c0 + 64 * hx + 4 * i4 + x) * 4u;
                    sb[i4][x] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sbr, co, 0, 0));
                    bi[i4][x] = -0.0f;          // adding it changes nothing, not even a zero's sign
                }
            if (LAYOUT == DENSE && p.bias) {
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        bi[i4][x] = __uint_as_float(
                            __builtin_amdgcn_raw_buffer_load_b32(bir, uint32_t(c0 + 64 * hx + 4 * i4 + x) * 4u, 0, 0));
            }
#pragma unroll
            for (int y = 0; y < MY; ++y) {
                typedef OutT o8 __attribute__((ext_vector_type(8)));
                u32x4 P[2];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    o8 v;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int i4 = 2 * hh + (c >> 2), x = c & 3;
                        v[c] = OutT(fmaf(float(acc[y][4 * hx + x][i4]) * sa[y], sb[i4][x], bi[i4][x]));
                    }
                    P[hh] = __builtin_bit_cast(u32x4, v);
                }
                // swap lane bit 0 with the 16-byte chunk, so that every store
                // instruction writes eight whole 128-byte lines
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint32_t a = P[0][d], b = P[1][d];
                    const uint32_t ax = uint32_t(__builtin_amdgcn_update_dpp(0, int(a), 0xB1, 0xF, 0xF, false));
                    const uint32_t bx = uint32_t(__builtin_amdgcn_update_dpp(0, int(b), 0xB1, 0xF, 0xF, false));
                    P[0][d] = odd ? bx : a;
                    P[1][d] = odd ? b : ax;
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int row = row_of((ln & 14) + hh, y);
                    const int col = c0 + 8 * (ln & 1) + 64 * hx;
                    const bool ok = (okh[hh] >> y) & 1;
                    const uint32_t off = (uint32_t(row) * uint32_t(p.N) + uint32_t(col)) * 2u;
                    const bool eight = ok && col + 8 <= cols;
                    if (dwords) __builtin_amdgcn_raw_buffer_store_b128(P[hh], dr, eight ? off : kOutside, 0, 2 /* nt */);
                    else if (eight) *reinterpret_cast<u32x4_at2*>(out + off) = P[hh];
                    if (cut && ok && !eight) {
#pragma unroll
                        for (int c = 0; c < 7; c += 2) {
                            if (col + c + 2 <= cols) *reinterpret_cast<uint32_at2*>(out + off + 2 * c) = P[hh][c / 2];
                            else if (col + c < cols) *reinterpret_cast<uint16_t*>(out + off + 2 * c) = uint16_t(P[hh][c / 2]);
                        }
                    }
                }
                GFG_SB();
            }
        }
        if (!have_next) break;
        cur = next;
        i = i_next;
    }
    GFG_WAITCNT(0, 0);
}

template <int LAYOUT, typename OutT>
__global__ __launch_bounds__(NTHREADS, 1) void int8_gemm256_kernel(I8Params p) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem0[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t smem1[STAGE];
    __shared__ uint32_t work[LAYOUT == DENSE ? 1 : CAND_MAX];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    GFG_LDS uint8_t* const buf0 = (GFG_LDS uint8_t*)smem0;
    GFG_LDS uint8_t* const buf1 = (GFG_LDS uint8_t*)smem1;
    if constexpr (LAYOUT != CONTIG) {
        int n256 = int((p.rows + 255) / 256), n192 = int((p.rows + 191) / 192);
        if (LAYOUT == MASKED) {                // of the rows that there are
            int a = 0, b = 0;
            for (int g = tid; g < p.G; g += NTHREADS) {
                const int mm = min(max(p.meta[g], 0), int(p.rows));
                a += (mm + 255) / 256;
                b += (mm + 191) / 192;
            }
            GFG_LDS int* const tmp = reinterpret_cast<GFG_LDS int*>(buf0);
            block_exclusive_scan<false>(a, tmp, lane, wave, &n256);
            block_exclusive_scan<false>(b, tmp, lane, wave, &n192);
        }
        const unsigned NT = unsigned(p.N + BN - 1) / BN, wgs = gridDim.x;
        const unsigned r256 = (unsigned(n256) * NT + wgs - 1) / wgs, r192 = (unsigned(n192) * NT + wgs - 1) / wgs;
        if (__builtin_amdgcn_readfirstlane(r192 * 7 < r256 * 8)) {
            walk_tiles<LAYOUT, 6, OutT>(p, buf0, buf1, work, tid, lane, wave);
            return;
        }
    }
    walk_tiles<LAYOUT, 8, OutT>(p, buf0, buf1, work, tid, lane, wave);
}

template <int LAYOUT>
void launch_t(const I8Params& p, unsigned grid, int out_dtype, hipStream_t s) {
    if (out_dtype == GFG_OUT_BF16)
        hipLaunchKernelGGL((int8_gemm256_kernel<LAYOUT, __bf16>), dim3(grid), dim3(NTHREADS), 0, s, p);
    else
        hipLaunchKernelGGL((int8_gemm256_kernel<LAYOUT, _Float16>), dim3(grid), dim3(NTHREADS), 0, s, p);
}

}  // namespace

int launch_int8_256(const I8Params& p, int layout, int out_dtype, hipStream_t s) {
    int cus = 0;
    if (int rc = device_cus(&cus)) return rc;
    const int64_t most = layout == CONTIG ? p.m_tiles : (p.rows + 191) / 192 * (layout == MASKED ? p.G : 1);
    const int64_t upper = most * ((p.N + BN - 1) / BN);
    unsigned grid = unsigned(upper < cus ? upper : cus);
    const int lim = grid_limit();
    if (lim > 0 && grid > unsigned(lim)) grid = unsigned(lim);
    const unsigned nx = unsigned(p.num_xcd);
    grid = (grid + nx - 1) / nx * nx;
    if (layout == DENSE) launch_t<DENSE>(p, grid, out_dtype, s);
    else if (layout == CONTIG) launch_t<CONTIG>(p, grid, out_dtype, s);
    else launch_t<MASKED>(p, grid, out_dtype, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

}  // namespace gfg
