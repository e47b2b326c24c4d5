// The dense FP8 (E4M3) product on 256 x 256 output tiles for gfx950 (MI355X): the
// launches of the linear layer and its gradients with enough of these tiles.
//
//   d[m, n] = sum_k a[m, k] b[n, k] (+ bias[n])
//
// with one E8M0 byte per row of `a` and 128 k and, for `b`, one per block of
// 128 x 128 or (BROW, the gradient of a weight) one per row and 128 k.
//
// Design: four wave64s, one per SIMD, each owning a 128 x 128 quarter of the
// tile: 256 accumulator registers (64 16x16 blocks) and 192 fragment registers.
// K goes in steps of 128, one v_mfma_scale_f32_16x16x128_f8f6f4 a block and step,
// through two 64 KB LDS stages filled by direct-to-LDS loads.  Alone on its SIMD,
// a wave's instruction order is the schedule, so every group of instructions is
// pinned in place: a step has two barriers, the first frees the rows of the
// stage whose fragments are already in registers, whose refill then runs under
// the step's own MFMAs, the second waits for the next stage.  The refills of a
// tile's last two steps load the next tile's first two stages, and its output
// stores go out after them, counted in the next tile's first wait.
//
// Sizes that are no multiple of the tile cost nothing inside the loop: rows
// past an operand's end and chunks past K have load offsets outside the buffer
// window, where the hardware returns zeros, and K is rounded up to an even
// number of steps.  A lane's four scale bytes are one load at any address, which
// starts lower for rows past the end and is shifted down.
//
// Measured: 4096 x 4096 x 16384 194-240 us by run (2290-2830 TFLOP/s), matrix pipes busy
// 62% of the cycles at 2.18 GHz, waves waiting 18% of theirs, the rest the wave's own
// LDS reads, loads and barriers; a step takes 1.5 us and more.  4096 x
// 7168 x 2304 70 us (448 tiles, 1.75 rounds), its weight's gradient 64, its tokens'
// 88 (144 tiles on 256 CUs).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_fp8_linear.h"
#include "gfg_internal.h"
#include "gfg_tile256.h"

namespace gfg {
namespace {

constexpr uint32_t kOutside = 0x80000000u;       // past every buffer window used here (all below 2^31 bytes)
constexpr int FIRST_HALF = 12;                   // a step's loads issued before its mid barrier (of 16)
typedef uint32_t u32_at1 __attribute__((aligned(1)));
typedef const __attribute__((address_space(1))) uint8_t* gbyte;      // (a pointer rebuilt from registers has lost its space)

// A wave's part of a tile: rows 128 wm .., columns 128 wn ...
struct Frags {
    int wave, wm, wn;
};
// The LDS offset of the 16-byte chunk lq of fragment 0's row in the first 64 of
// the operand's 128 rows w; computed from the lane index where it is used, so
// that it takes no register through the loop.  The row of fragment f is f ^ (l16
// & 1) of four, so its offset differs in bits 7 and 8, and chunk lq + 4's in bit 6.
__device__ __forceinline__ int frag_base(int w) {
    const int ln = lane_now(), l16 = ln & 15;
    return swz_a(w * 128 + 4 * l16, ln >> 4) ^ ((l16 & 1) << 7);
}
__device__ __forceinline__ int frag_at(int e, int y, bool hi) { return (e ^ ((y & 3) << 7) ^ (hi ? 64 : 0)) + (y >> 2) * 64 * BK; }

// What the refills of one tile read.
struct Source {
    __amdgpu_buffer_rsrc_t a, b;
    const uint8_t* sb_row;   // blocks: the scale bytes (all K blocks) of this wave's 128 columns
    int row0, n0;
};

__device__ __forceinline__ TileInfo tile_of(const F8Params& p, int mr, int nt) {
    TileInfo t;
    t.g = 0;
    t.row0 = __builtin_amdgcn_readfirstlane(mr * BM);
    t.lim = __builtin_amdgcn_readfirstlane(int(p.rows - t.row0 < BM ? p.rows - t.row0 : BM));
    t.n0 = __builtin_amdgcn_readfirstlane(nt * BN);
    return t;
}

template <bool BROW>
__device__ __forceinline__ Source source_of(const F8Params& p, const TileInfo& t, int wn) {
    const int cols = min(BN, p.N - t.n0);
    Source s;
    s.a = make_rsrc(p.a + int64_t(t.row0) * p.K, uint32_t(t.lim) * uint32_t(p.K));
    s.b = make_rsrc(p.b + int64_t(t.n0) * p.K, uint32_t(cols) * uint32_t(p.K));
    // (a tile may end before its second 128 columns)
    s.sb_row = BROW ? nullptr : uniform_ptr(p.b_scale + int64_t(min(t.n0 / 128 + wn, (p.N - 1) / 128)) * p.KB);
    s.row0 = t.row0;
    s.n0 = t.n0;
    return s;
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

// Load chunk c (0..7: A's, 8..15: B's) of a stage: 32 (c & 7) rows further on.
__device__ __forceinline__ void refill(const Source& r, uint32_t off, int K, GFG_LDS uint8_t* dst, int wave, int c) {
    asm volatile("" : "+v"(off));   // added per chunk, not eight offsets held live
    const int j = c & 7;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(c < 8 ? r.a : r.b, (GFG_LDS void*)(dst + (j * WAVES + wave) * 1024), 16,
                                             off + uint32_t(32 * j) * uint32_t(K), 0, 0, 0);
}

// The scale bytes of one stage: four rows of each 64-row half of A, and of B's.
template <bool BROW>
struct Scales {
    uint32_t a[2], b[2];     // blocks: b[0] the word of the block's byte, b[1] its shift (scalar registers)
};

// Row (of `total` >= 4) of the lane's bytes in half h of a wave's 128 rows; and
// where their load starts.
__device__ __forceinline__ int scale_row(int first, int h) { return first + 64 * h + 4 * (lane_now() & 15); }
__device__ __forceinline__ uint32_t scale_load(const uint8_t* base, int row, int total) {
    return *(const __attribute__((address_space(1))) u32_at1*)((gbyte)base + uint32_t(min(row, total - 4)));
}
__device__ __forceinline__ int scale_down(uint32_t raw, int row, int total) {
    const int by = row - (total - 4);
    return by <= 0 ? int(raw) : by < 4 ? int(raw >> (8 * by)) : 0;
}

// Vector-memory operations: 2, or 4 with BROW (the blocks' bytes come through the scalar cache).
template <bool BROW>
__device__ __forceinline__ void load_scales(const F8Params& p, const Source& r, const Frags& L, int kb, Scales<BROW>& s) {
    const int ks = min(kb, p.KB - 1);
    const uint8_t* const a = uniform_ptr(p.a_scale + ks * p.ld_a);
#pragma unroll
    for (int h = 0; h < 2; ++h) s.a[h] = scale_load(a, scale_row(r.row0 + L.wm * 128, h), int(p.rows));
    if constexpr (BROW) {
        const uint8_t* const b = uniform_ptr(p.b_scale + ks * p.ld_b);
#pragma unroll
        for (int h = 0; h < 2; ++h) s.b[h] = scale_load(b, scale_row(r.n0 + L.wn * 128, h), p.N);
    } else {
        s.b[0] = uint32_t(load_scale_word(r.sb_row, ks));
        s.b[1] = 8u * __builtin_amdgcn_readfirstlane(uint32_t(reinterpret_cast<uintptr_t>(r.sb_row) + uintptr_t(ks)) & 3u);
    }
}

__device__ __forceinline__ v8i join(u32x4 l, u32x4 h) {
    return __builtin_bit_cast(v8i, __builtin_shufflevector(l, h, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int SB>
__device__ __forceinline__ v4f mfma_b(const v8i& b, const v8i& a, const v4f& c, int sb, int y, int sa) {
    switch (y & 3) {   // the scale bytes (op_sel) must be constants
        case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, SB, sb, 0, sa);
        case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, SB, sb, 1, sa);
        case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, SB, sb, 2, sa);
        default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, SB, sb, 3, sa);
    }
}
template <bool BROW>
__device__ __forceinline__ v4f mfma(const v8i& b, const v8i& a, const v4f& c, int x, const int (&sb)[2], int y, int sa) {
    if constexpr (!BROW) return mfma_b<0>(b, a, c, sb[0], y, sa);
    switch (x & 3) {
        case 0: return mfma_b<0>(b, a, c, sb[x >> 2], y, sa);
        case 1: return mfma_b<1>(b, a, c, sb[x >> 2], y, sa);
        case 2: return mfma_b<2>(b, a, c, sb[x >> 2], y, sa);
        default: return mfma_b<3>(b, a, c, sb[x >> 2], y, sa);
    }
}

// One step k: stage k in `cur` (its B region also as `cur_b`), stage k+1 in
// `nxt`; stage kr (of the tile that `rf` reads) refills `cur`, and its scales
// replace stage k's.  On entry af[0..3] and bc hold stage k's A fragments 0..3
// and B fragments; row0 and n0 are those of stage k's tile.  VMWAIT: vector-
// memory operations issued after stage k+1's last load that may be in flight at
// the mid barrier.
template <int VMWAIT, bool BROW>
__device__ __forceinline__ void step(const F8Params& p, const Frags& L, int row0, int n0, GFG_LDS uint8_t* __restrict__ cur,
                                     GFG_LDS uint8_t* __restrict__ cur_b, GFG_LDS uint8_t* __restrict__ nxt, int kr, const Source& rf,
                                     v4f (&acc)[8][8], v8i (&af)[8], v8i (&bc)[8], v8i (&bn)[8], Scales<BROW>& s) {
    GFG_SB();
    GFG_WAITCNT(63, 0);
    __builtin_amdgcn_s_barrier();
    GFG_SB();
    int sa[2], sb[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        sa[h] = scale_down(s.a[h], scale_row(row0 + L.wm * 128, h), int(p.rows));
        if constexpr (BROW) sb[h] = scale_down(s.b[h], scale_row(n0 + L.wn * 128, h), p.N);
    }
    if constexpr (!BROW) sb[0] = int((s.b[0] >> s.b[1]) & 0xFFu);
    const uint32_t off = stage_offset(L.wave, kr, p.K);
    GFG_SB();
    {
        u32x4 r[8];
        const int e = frag_base(L.wm);
#pragma unroll
        for (int m = 0; m < 32; ++m) {
            const int y = m >> 3, x = m & 7;
            acc[y][x] = mfma<BROW>(bc[x], af[y], acc[y][x], x, sb, y, sa[0]);
            GFG_SB();
            if (m < 8) {
                const int yy = 4 + (m >> 1);
                r[m] = lds16(cur, frag_at(e, yy, m & 1));
                GFG_SB();
            }
            if (m >= 8 && !(m & 1)) {
                const int q = (m - 8) >> 1;   // 0..11: A chunks 0, 1, 4, 5 (fragment rows 0..3), then B's
                if (q < 4) refill(rf, off, p.K, cur, L.wave, (q & 1) + 4 * (q >> 1));
                else refill(rf, off, p.K, cur_b, L.wave, 8 + q - 4);
                GFG_SB();
            }
        }
#pragma unroll
        for (int f = 0; f < 4; ++f) af[4 + f] = join(r[2 * f], r[2 * f + 1]);
    }
    GFG_WAITCNT(VMWAIT, 0);
    __builtin_amdgcn_s_barrier();
    GFG_SB();
    {
        u32x4 r[24];
        const int ea = frag_base(L.wm), eb = A_BYTES + frag_base(L.wn);
#pragma unroll
        for (int m = 0; m < 32; ++m) {
            const int y = 4 + (m >> 3), x = m & 7;
            acc[y][x] = mfma<BROW>(bc[x], af[y], acc[y][x], x, sb, y, sa[1]);
            GFG_SB();
            if ((m & 7) == 1) refill(rf, off, p.K, cur, L.wave, 2 + ((m >> 3) & 1) + 4 * (m >> 4));   // chunks 2, 3, 6, 7
            if (m < 16) {
                const int xx = m >> 1;
                r[m] = lds16(nxt, frag_at(eb, xx, m & 1));
            } else if (m < 24) {
                const int yy = (m - 16) >> 1;
                r[m] = lds16(nxt, frag_at(ea, yy, m & 1));
            }
            GFG_SB();
        }
#pragma unroll
        for (int f = 0; f < 8; ++f) bn[f] = join(r[2 * f], r[2 * f + 1]);
#pragma unroll
        for (int f = 0; f < 4; ++f) af[f] = join(r[16 + 2 * f], r[17 + 2 * f]);
    }
    load_scales<BROW>(p, rf, L, kr, s);
    GFG_SB();
}

// The bit that takes a store past its window where the column is past the end
// (not a choice of offsets, which the compiler may turn into two stores behind branches).
__device__ __forceinline__ uint32_t past(int col, int cols) { return uint32_t(cols - 1 - col) & 0x80000000u; }

// BIAS: there is one; ADD: d is added to (32 bits); WHOLE: N is a multiple of 8,
// so that every chunk of eight columns is inside a row or past it.
template <bool BROW, bool BIAS, bool ADD, bool WHOLE, typename OutT>
__global__ __launch_bounds__(NTHREADS, 1) void fp8_dense256_kernel(F8Params p) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem0[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t smem1[STAGE];
    __shared__ __attribute__((aligned(1024))) float bias_smem[BIAS ? 2 * BN : 1];   // of this tile's columns and the next one's
    constexpr int SL = BROW ? 4 : 2;                       // scale loads a stage
    constexpr int STORES = sizeof(OutT) == 4 ? 64 : 32;    // of a tile, by every wave
    constexpr int STEADY = SL + FIRST_HALF;
    constexpr int BOUNDARY = STEADY + STORES + (BIAS ? 1 : 0);
    constexpr int FIRST = BOUNDARY < 62 ? BOUNDARY : 62;   // (63 would be no wait)

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GFG_LDS uint8_t* const buf0 = (GFG_LDS uint8_t*)smem0;
    GFG_LDS uint8_t* const buf1 = (GFG_LDS uint8_t*)smem1;
    const unsigned MT = unsigned((p.rows + BM - 1) / BM), NT = unsigned(p.N + BN - 1) / BN;
    TileOrder order;
    order.init(MT * NT, p.num_xcd);
    order.x_start = __builtin_amdgcn_readfirstlane(order.x_start);
    order.x_count = __builtin_amdgcn_readfirstlane(order.x_count);
    order.slot = __builtin_amdgcn_readfirstlane(order.slot);
    order.slots = __builtin_amdgcn_readfirstlane(order.slots);
    const unsigned gm = p.group_m > 0 ? unsigned(p.group_m) : 4u;
    unsigned i = order.slot;
    if (i >= order.x_count) return;

    Frags L;
    L.wave = wave;
    L.wm = wave >> 1;
    L.wn = wave & 1;
    const int KB2 = (p.KB + 1) & ~1;       // an even number of steps; those past K add zeros
    __builtin_assume(KB2 >= 2);
    int mr, nt;
    order.item(i, gm, NT, MT, &mr, &nt);
    TileInfo cur = tile_of(p, mr, nt);
    Source rf = source_of<BROW>(p, cur, L.wn);

    v4f acc[8][8];
    v8i af[8], bf0[8], bf1[8];
    Scales<BROW> s0, s1;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint32_t off = stage_offset(wave, s, p.K);
#pragma unroll
        for (int c = 0; c < 16; ++c) refill(rf, off, p.K, (s ? buf1 : buf0) + (c < 8 ? 0 : A_BYTES), wave, c);
    }
    load_scales<BROW>(p, rf, L, 0, s0);
    load_scales<BROW>(p, rf, L, 1, s1);
    // everything has landed, so the first tile's first wait, which counts the
    // stores of a tile before it, has nothing left to wait for
    GFG_WAITCNT(0, 15);
    __builtin_amdgcn_s_barrier();
    const int ea = frag_base(L.wm), eb = A_BYTES + frag_base(L.wn);
#pragma unroll
    for (int y = 0; y < 4; ++y)
        af[y] = join(lds16(buf0, frag_at(ea, y, false)), lds16(buf0, frag_at(ea, y, true)));
#pragma unroll
    for (int x = 0; x < 8; ++x)
        bf0[x] = join(lds16(buf0, frag_at(eb, x, false)), lds16(buf0, frag_at(eb, x, true)));

    int turn = 0;
    while (true) {
        if constexpr (BIAS) {
            // each wave's 64 columns, by a direct-to-LDS load like the stages'; it has
            // landed everywhere by the second step's mid barrier
            const __amdgpu_buffer_rsrc_t br = make_rsrc(p.bias + cur.n0, uint32_t(min(BN, p.N - cur.n0)) * 4u);
            GFG_SB();
            __builtin_amdgcn_raw_ptr_buffer_load_lds(br, (GFG_LDS void*)((GFG_LDS float*)bias_smem + turn * BN + wave * 64), 4,
                                                     uint32_t(wave * 64 + lane_now()) * 4u, 0, 0, 0);
            GFG_SB();
        }
#pragma unroll
        for (int y = 0; y < 8; ++y)
#pragma unroll
            for (int x = 0; x < 8; ++x) acc[y][x] = v4f{};
        i = __builtin_amdgcn_readfirstlane(i);
        const unsigned i_next = i + order.slots;
        const bool have_next = i_next < order.x_count;
        TileInfo next = cur;
        if (have_next) {
            int mr2, nt2;
            order.item(i_next, gm, NT, MT, &mr2, &nt2);
            next = tile_of(p, mr2, nt2);
        }
        // Step k refills with stage k + 2; from step KB2 - 2 on with the next
        // tile's stage k + 2 - KB2, or, on the last tile, with nothing (a stage
        // past K lies outside the window).
        const int wrap = __builtin_amdgcn_readfirstlane(have_next ? KB2 : 0);
        auto stage_of = [&](int k) { return __builtin_amdgcn_readfirstlane(k + 2 < KB2 ? k + 2 : k + 2 - wrap); };
        if (KB2 == 2 && have_next) rf = source_of<BROW>(p, next, L.wn);
        step<FIRST, BROW>(p, L, cur.row0, cur.n0, buf0, buf0 + A_BYTES, buf1, stage_of(0), rf, acc, af, bf0, bf1, s0);
        step<STEADY, BROW>(p, L, cur.row0, cur.n0, buf1, buf1 + A_BYTES, buf0, stage_of(1), rf, acc, af, bf1, bf0, s1);
        for (int kb = 2; kb < KB2; kb += 2) {
            if (kb + 2 == KB2 && have_next) rf = source_of<BROW>(p, next, L.wn);
            step<STEADY, BROW>(p, L, cur.row0, cur.n0, buf0, buf0 + A_BYTES, buf1, stage_of(kb), rf, acc, af, bf0, bf1, s0);
            step<STEADY, BROW>(p, L, cur.row0, cur.n0, buf1, buf1 + A_BYTES, buf0, stage_of(kb + 1), rf, acc, af, bf1, bf0, s1);
        }

        // ---- epilogue.  Lane (l16, lq) holds, for each y, output row
        // 128 wm + 64 (y >> 2) + 4 l16 + (y & 3), and for each column half hx
        // columns 128 wn + 64 hx + 16 lq + 4 i + x in acc[y][4 hx + x][i].
        const int ln = lane_now();
        const int cols = min(BN, p.N - cur.n0);
        OutT* const out = static_cast<OutT*>(p.d) + int64_t(cur.row0) * p.N + cur.n0;
        const __amdgpu_buffer_rsrc_t dr = make_rsrc(out, uint32_t(cur.lim) * uint32_t(p.N) * uint32_t(sizeof(OutT)));
        const int c0 = L.wn * 128 + 16 * (ln >> 4);
        const int r0 = L.wm * 128 + 4 * (ln & 15);
        // the bias of columns c0 + 64 hx + 4 q .. +3
        auto bias4 = [&](int hx, int q) {
            if constexpr (BIAS) return reinterpret_cast<const GFG_LDS v4f*>((const GFG_LDS float*)bias_smem + turn * BN + c0)[16 * hx + q];
            else return v4f{};
        };
        // Whole chunks of eight columns go out as buffer stores, a fixed number by
        // every wave: a row or a chunk past the end falls outside the window.
        if constexpr (WHOLE && sizeof(OutT) == 4) {
            // two rows' 16 columns at a time; with ADD their old values are loaded together
#pragma unroll
            for (int hx = 0; hx < 2; ++hx)
#pragma unroll
                for (int y0 = 0; y0 < 8; y0 += 2) {
                    auto at = [&](int y, int q) {
                        const int row = r0 + 64 * (y >> 2) + (y & 3), col = c0 + 64 * hx + 4 * q;
                        return ((uint32_t(row) * uint32_t(p.N) + uint32_t(col)) * 4u) | past(col, cols);
                    };
                    u32x4 old[2][4];
                    if constexpr (ADD) {
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int q = 0; q < 4; ++q) old[y][q] = __builtin_amdgcn_raw_buffer_load_b128(dr, at(y0 + y, q), 0, 0);
                        GFG_SB();
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const v4f* const a = &acc[y0 + y][4 * hx];
                            v4f v = {a[0][q], a[1][q], a[2][q], a[3][q]};
                            if constexpr (ADD) v += __builtin_bit_cast(v4f, old[y][q]);
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), dr, at(y0 + y, q), 0, 0);
                        }
                    GFG_SB();
                }
        } else if constexpr (WHOLE) {
#pragma unroll
            for (int hx = 0; hx < 2; ++hx) {
                v4f b[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) b[q] = bias4(hx, q);
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    // Swapping lane bit 0 with the chunk hands slot h of lane l16 row
                    // 4 ((l16 & ~1) | h) and chunk 2 lq + (l16 & 1), so that every store
                    // instruction writes eight whole 128-byte lines.
                    typedef OutT out8 __attribute__((ext_vector_type(8)));
                    typedef float f8v __attribute__((ext_vector_type(8)));
                    const bool odd = (ln & 1) != 0;
                    u32x4 P[2];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const v4f v0 = acc[y][4 * hx], v1 = acc[y][4 * hx + 1], v2 = acc[y][4 * hx + 2], v3 = acc[y][4 * hx + 3];
                        f8v v = {v0[2 * hh], v1[2 * hh], v2[2 * hh], v3[2 * hh],
                                 v0[2 * hh + 1], v1[2 * hh + 1], v2[2 * hh + 1], v3[2 * hh + 1]};
                        if constexpr (BIAS) v += __builtin_shufflevector(b[2 * hh], b[2 * hh + 1], 0, 1, 2, 3, 4, 5, 6, 7);
                        P[hh] = __builtin_bit_cast(u32x4, __builtin_convertvector(v, out8));
                    }
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
                        const int row = L.wm * 128 + 4 * ((ln & 14) + hh) + 64 * (y >> 2) + (y & 3);
                        const int col = c0 + 8 * (ln & 1) + 64 * hx;
                        const uint32_t off = ((uint32_t(row) * uint32_t(p.N) + uint32_t(col)) * 2u) | past(col, cols);
                        __builtin_amdgcn_raw_buffer_store_b128(P[hh], dr, off, 0, 2 /* nt */);
                    }
                    GFG_SB();
                }
            }
        } else {
            // rows that start anywhere: vectors of the elements' alignment, single
            // elements at the end of a row
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const int row = r0 + 64 * (y >> 2) + (y & 3);
#pragma unroll
                for (int hx = 0; hx < 2; ++hx)
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        typedef OutT vec __attribute__((ext_vector_type(8), aligned(sizeof(OutT))));
                        const int col = c0 + 64 * hx + 4 * q;
                        OutT* const at = out + int64_t(row) * p.N + col;
                        vec v;
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = OutT(acc[y][4 * hx + (j & 3)][q + (j >> 2)] + (BIAS ? bias4(hx, q + (j >> 2))[j & 3] : 0.0f));
                        if (row < cur.lim) {
                            if (col + 8 <= cols) {
                                *reinterpret_cast<vec*>(at) = v;
                            } else {
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    if (col + j < cols) at[j] = v[j];
                            }
                        }
                        GFG_SB();
                    }
            }
            GFG_WAITCNT(0, 15);                            // (not a fixed number of them)
        }
        turn ^= 1;
        if (!have_next) break;
        cur = next;
        i = i_next;
    }
    GFG_WAITCNT(0, 0);
}

}  // namespace

bool fp8_256_fits(const F8Params& p, int out_dtype) {
    return p.rows >= 4 && p.N >= 4 && p.rows <= (1 << 30) && p.N <= (out_dtype == GFG_OUT_F32 ? 1 << 20 : 1 << 21);
}

// brow: N a multiple of 8 and no bias; otherwise nothing is added to (d has 16 bits).
int launch_fp8_256(const F8Params& p, bool brow, int out_dtype, hipStream_t s) {
    int cus = 0;
    if (int rc = device_cus(&cus)) return rc;
    const int64_t tiles = (p.rows + BM - 1) / BM * ((p.N + BN - 1) / BN);
    unsigned grid = unsigned(tiles < cus ? tiles : cus);
    const int lim = grid_limit();
    if (lim > 0 && grid > unsigned(lim)) grid = unsigned(lim);
    const unsigned nx = unsigned(p.num_xcd);
    grid = (grid + nx - 1) / nx * nx;
    auto go = [&](auto* kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(NTHREADS), 0, s, p); };
    auto dense = [&](auto one) {
        typedef decltype(one) T;
        if (p.N % 8) go(p.bias ? fp8_dense256_kernel<false, true, false, false, T> : fp8_dense256_kernel<false, false, false, false, T>);
        else go(p.bias ? fp8_dense256_kernel<false, true, false, true, T> : fp8_dense256_kernel<false, false, false, true, T>);
    };
    if (!brow && out_dtype == GFG_OUT_BF16) dense(__bf16{});
    else if (!brow) dense(_Float16{});
    else if (out_dtype == GFG_OUT_BF16) go(fp8_dense256_kernel<true, false, false, true, __bf16>);
    else if (out_dtype == GFG_OUT_F16) go(fp8_dense256_kernel<true, false, false, true, _Float16>);
    else go(p.accumulate ? fp8_dense256_kernel<true, false, true, true, float> : fp8_dense256_kernel<true, false, false, true, float>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

}  // namespace gfg
