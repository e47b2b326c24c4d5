// 8-bit integer matrix product with one scale per token and per output
// channel, and the token quantizer that makes its operand, for gfx950 (MI355X).
//
//   q[m, k] = rint(x[m, k] * (127 / amax[m])),  s[m] = amax[m] / 127,
//   amax[m] = max(max_k |x[m, k]|, 2^-100)
//   d[m, n] = (sum_k a[m, k] b[n, k]) * a_scale[m] * b_scale[n] (+ bias[n])
//
// The sums are 32-bit integers, which v_mfma_i32_16x16x64_i8 accumulates
// exactly (K < 2^17, so |sum| <= 2^14 K < 2^31), so neither the order of the
// K steps nor a split of K changes a bit; the two scales are applied in fp32
// and the output is rounded once.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gfg.h"
#include "gfg_device.h"
#include "gfg_int8.h"
#include "gfg_internal.h"

namespace gfg {
namespace {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------ token quantizer
//
// One pass over memory: a row's 16-byte chunks stay in registers between the
// maximum and the encoding, HELD a lane (longer rows read the rest again, from
// the cache).  LPR lanes share a row: a wave up to 2048 elements, two waves up
// to 3 * 1024, four past that; with more than one, the maximum crosses the waves
// through LDS.  Bound by the copy rate (5.0 TB/s).  Measured, us on one, two and
// four waves a row: bf16 32768 x 2048 40.8 (4.9 TB/s of reads and writes), 41.1,
// 49.5; 32768 x 2304 45.6, 47.9, 54.7 (f32 73.0, 68.8, 67.8); 16384 x 3584 38.1, 36.0,
// 34.3 (f32 66.2, 54.5, 50.0); 8192 x 7168 42.4, 40.9, 33.6 (5.2 TB/s).  4096 x 16384
// on four: 41.2, with half of the row held 45.0 (f32 70.3 and 80.3).
template <typename T> struct Chunk;            // 8 elements of a row
template <> struct Chunk<__bf16> {
    u32x4 w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) { w = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0); }
    __device__ __forceinline__ void load(const __bf16* p) { w = *reinterpret_cast<const u32x4*>(p); }
    __device__ __forceinline__ float at(int i) const {
        return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    }
};
template <> struct Chunk<_Float16> {
    u32x4 w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) { w = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0); }
    __device__ __forceinline__ void load(const _Float16* p) { w = *reinterpret_cast<const u32x4*>(p); }
    __device__ __forceinline__ float at(int i) const {
        return float(__builtin_bit_cast(_Float16, uint16_t(w[i >> 1] >> (16 * (i & 1)))));
    }
};
template <> struct Chunk<float> {
    u32x4 w[2];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
        w[1] = __builtin_amdgcn_raw_buffer_load_b128(r, at + 16, 0, 0);
    }
    __device__ __forceinline__ void load(const float* p) {
        w[0] = reinterpret_cast<const u32x4*>(p)[0];
        w[1] = reinterpret_cast<const u32x4*>(p)[1];
    }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i >> 2][i & 3]); }
};

// Maximum of the magnitude bits: for finite floats the integer order is the
// order of the magnitudes, and an infinity or a NaN lands above all of them.
template <typename T>
__device__ __forceinline__ uint32_t chunk_amax(const Chunk<T>& c) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(c.at(i)) & 0x7FFFFFFFu);
    return m;
}

// Eight codes; |x * r| <= 127 up to one rounding, so rint never leaves [-127, 127].
template <typename T>
__device__ __forceinline__ u32x2 chunk_encode(const Chunk<T>& c, float r) {
    u32x2 o = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int v = int(__builtin_rintf(c.at(i) * r));
        o[i >> 2] |= uint32_t(v & 0xFF) << (8 * (i & 3));
    }
    return o;
}

// The scale of a row with magnitude bits ab, and the factor 127 / amax of its codes.
__device__ __forceinline__ void row_scale(uint32_t ab, float* scale, float* r) {
    if (ab >= 0x7F800000u) {                   // a NaN or an infinity: no scale, codes 0
        *scale = __uint_as_float(0x7FC00000u);
        *r = 0.0f;
    } else {
        const float amax = fmaxf(__uint_as_float(ab), 0x1p-100f);
        *scale = amax / 127.0f;
        *r = 127.0f / amax;
    }
}

template <typename T, int LPR, int HELD>
__global__ __launch_bounds__(LPR == 64 ? 256 : LPR) void quant_token_kernel(const T* __restrict__ x, uint8_t* __restrict__ q,
                                                         float* __restrict__ scale, int64_t M, int K) {
    constexpr int RPB = LPR == 64 ? 4 : 1;      // rows per workgroup
    __shared__ uint32_t part[2][LPR / 64];     // in turn: a row's maxima are read while the next row's are written
    const int lane = threadIdx.x % LPR, chunks = K / 8;
    int turn = 0;
    for (int64_t m = int64_t(blockIdx.x) * RPB + threadIdx.x / LPR; m < M; m += int64_t(gridDim.x) * RPB, turn ^= 1) {
        const T* row = x + m * K;
        Chunk<T> held[HELD];
        uint32_t ab = 0;
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            if (lane + j * LPR < chunks) held[j].load(row + (lane + j * LPR) * 8);
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            if (lane + j * LPR < chunks) ab = max(ab, chunk_amax(held[j]));
        for (int c = lane + HELD * LPR; c < chunks; c += LPR) {
            Chunk<T> t;
            t.load(row + c * 8);
            ab = max(ab, chunk_amax(t));
        }
        ab = wave_reduce(ab, [](uint32_t a, uint32_t b) { return max(a, b); });
        if constexpr (LPR > 64) {              // (the workgroup's lanes share the row: all of them are here)
            if ((threadIdx.x & 63) == 0) part[turn][threadIdx.x >> 6] = ab;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < LPR / 64; ++w) ab = max(ab, part[turn][w]);
        }
        float s, r;
        row_scale(ab, &s, &r);
        if (lane == 0) scale[m] = s;
        uint8_t* out = q + m * K;
        const bool bad = r == 0.0f;            // 0 * infinity would be NaN
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            if (lane + j * LPR < chunks)
                *reinterpret_cast<u32x2*>(out + (lane + j * LPR) * 8) = bad ? u32x2{0u, 0u} : chunk_encode(held[j], r);
        for (int c = lane + HELD * LPR; c < chunks; c += LPR) {
            Chunk<T> t;
            t.load(row + c * 8);
            *reinterpret_cast<u32x2*>(out + c * 8) = bad ? u32x2{0u, 0u} : chunk_encode(t, r);
        }
    }
}

template <typename T, int LPR, int HELD>
void launch_quant_rows(const void* x, uint8_t* q, float* scale, int64_t M, int K, hipStream_t s) {
    constexpr int64_t most = 1 << 22;          // workgroups; each walks on where there are more rows
    constexpr int threads = LPR == 64 ? 256 : LPR;
    const int64_t wgs = (M * LPR + threads - 1) / threads;
    hipLaunchKernelGGL((quant_token_kernel<T, LPR, HELD>), dim3(unsigned(wgs < most ? wgs : most)), dim3(threads), 0, s,
                       static_cast<const T*>(x), q, scale, M, K);
}

template <typename T>
void launch_quant(const void* x, uint8_t* q, float* scale, int64_t M, int K, hipStream_t s) {
    if (K <= 64 * 8 * 4) launch_quant_rows<T, 64, 4>(x, q, scale, M, K, s);
    else if (K <= 128 * 8 * 3) launch_quant_rows<T, 128, 3>(x, q, scale, M, K, s);
    else if (K <= 256 * 8 * 4) launch_quant_rows<T, 256, 4>(x, q, scale, M, K, s);
    else launch_quant_rows<T, 256, 8>(x, q, scale, M, K, s);
}

// ------------------------------------------------------------------ tiled product
//
// TM x TN output tiles, WM x WN waves, K in steps of 128 bytes through S LDS
// stages filled by direct-to-LDS loads: S - 1 stages are in flight while one
// is consumed, and a step has one barrier (a wave that passes it has seen
// every wave finish the previous step, whose buffer the new loads go to).
// These are the launches with too few 256 x 256 tiles, whose time is the
// latency of a tile's first loads plus a chain of steps, so depth matters
// more than the bytes per step (with one stage ahead, the first form of this
// kernel, 1024 x 4096 x 4096 took 1.6 times as long, 512 x 4096 x 4096 twice; they
// take 23.5 and 17.5 us).  LDS row R (128 bytes)
// holds its 16-byte chunks XOR-swizzled by R & 7, so that the 16 rows that a
// fragment read touches spread over all banks.  Rows past the operand's end and chunks past K lie
// outside the buffer window, where the hardware returns zeros, so no size
// needs its own path: zeros add nothing to an integer sum.
constexpr int TK = 128;
constexpr uint32_t kOutside = 0x80000000u;     // past every buffer window used here (all below 2^31 bytes)

// One output element row piece: columns n .. n+3 of a row, from the integer sums.
template <typename OutT>
__device__ __forceinline__ void store4(OutT* row, int n, int N, const float (&v)[4]) {
    typedef OutT o4 __attribute__((ext_vector_type(4), aligned(2)));      // (rows start anywhere where N is odd)
    if (n + 4 <= N) {
        *reinterpret_cast<o4*>(row + n) = o4{OutT(v[0]), OutT(v[1]), OutT(v[2]), OutT(v[3])};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N) row[n + i] = OutT(v[i]);
    }
}

template <int LAYOUT, int TM, int TN, int S, int WM, int WN, typename OutT>
__device__ __forceinline__ void ring_tile(const I8Params& p, unsigned w) {
    constexpr int WAVES = WM * WN, BYTES = (TM + TN) * TK;
    constexpr int PER = BYTES / 1024 / WAVES;      // 1 KB loads per wave and stage
    constexpr int RB = TM / WM / 16, CB = TN / WN / 16;
    static_assert(S == 4 && BYTES % (1024 * WAVES) == 0 && TM % (8 * WAVES) == 0, "stage shape");
    // an array for each stage: the compiler then knows that reading one need
    // not wait for the loads into another
    __shared__ __attribute__((aligned(1024))) uint8_t s0[BYTES], s1[BYTES], s2[BYTES], s3[BYTES];
    GFG_LDS uint8_t* const buf[S] = {(GFG_LDS uint8_t*)s0, (GFG_LDS uint8_t*)s1, (GFG_LDS uint8_t*)s2, (GFG_LDS uint8_t*)s3};
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    // tiles in ranges, one for each XCD (the hardware deals workgroup w to XCD
    // w % num_xcd), row tiles first, so that a B panel stays in one L2
    const unsigned nx = unsigned(p.num_xcd), x = w % nx, per = p.tiles / nx, rem = p.tiles % nx;
    const unsigned item = x * per + min(x, rem) + w / nx;
    const int mt = int(item % unsigned(p.m_tiles)), n0 = int(item / unsigned(p.m_tiles)) * TN;
    int g = 0, row0, lim;
    int64_t region = 0;
    if (LAYOUT == MASKED) {
        g = mt / p.tiles_per_group;
        row0 = (mt - g * p.tiles_per_group) * TM;
        int mm = p.meta[g];
        mm = mm < 0 ? 0 : (mm > p.rows ? int(p.rows) : mm);
        lim = min(TM, mm - row0);
        region = int64_t(g) * p.rows;
    } else {
        row0 = mt * TM;
        lim = int(p.rows - row0 < TM ? p.rows - row0 : TM);
        if (LAYOUT == CONTIG) {
            g = p.meta[row0 & ~127];               // the expert of the aligned 128 rows
            if (g < 0 || g >= p.G) return;
        }
    }
    if (lim <= 0) return;
    g = __builtin_amdgcn_readfirstlane(g);
    lim = __builtin_amdgcn_readfirstlane(lim);
    const int64_t arow = region + row0;
    const int ncols = min(TN, p.N - n0);
    const auto ra = make_rsrc(p.a + arow * p.K, uint32_t(lim) * uint32_t(p.K));
    const auto rb = make_rsrc(p.b + (int64_t(g) * p.N + n0) * p.K, uint32_t(ncols) * uint32_t(p.K));

    // load j of a wave: LDS rows 8 (WAVES j + wave) .. +7 of the stage (A's TM
    // rows, then B's); lane i writes physical chunk i & 7 of row i >> 3 of
    // them, the logical chunk (i & 7) ^ (i >> 3)
    const int kc = ((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t src0 = uint32_t(8 * wave + (lane >> 3)) * uint32_t(p.K) + uint32_t(kc);
    auto issue = [&](GFG_LDS uint8_t* dst, int kb) {
        const uint32_t base = kb * TK + kc < p.K ? src0 + uint32_t(kb) * TK : kOutside;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            constexpr int A_LOADS = TM / 8 / WAVES;
            const int jr = j < A_LOADS ? j : j - A_LOADS;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(j < A_LOADS ? ra : rb, (GFG_LDS void*)(dst + (WAVES * j + wave) * 1024), 16,
                                                     base + uint32_t(8 * WAVES * jr) * uint32_t(p.K), 0, 0, 0);
        }
    };
    const int wm = (wave / WN) * (TM / WM), wn = (wave % WN) * (TN / WN);
    auto frag = [&](GFG_LDS uint8_t* src, int row, int chunk) {
        return *reinterpret_cast<GFG_LDS v4i*>(src + (row + l16) * TK + ((chunk ^ (l16 & 7)) << 4));
    };
    v4i acc[RB][CB] = {};                          // [row block][column block]
    const int KB = (p.K + TK - 1) / TK;
#pragma unroll
    for (int j = 0; j < S - 1; ++j) issue(buf[j], j);
    // one step on stage j's buffer: stage kb has landed here, and this wave's
    // reads of the stage before it are done; after the barrier, everyone's
    auto step = [&](GFG_LDS uint8_t* cur, GFG_LDS uint8_t* freed, int kb) {
        __builtin_amdgcn_sched_barrier(0);
        GFG_WAITCNT((S - 2) * PER, 15);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue(freed, kb + S - 1);                  // a stage past K loads zeros
        __builtin_amdgcn_sched_barrier(0);
        v4i af[2][RB], bf[2][CB];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int f = 0; f < RB; ++f) af[h][f] = frag(cur, wm + 16 * f, 4 * h + lq);
#pragma unroll
            for (int f = 0; f < CB; ++f) bf[h][f] = frag(cur + TM * TK, wn + 16 * f, 4 * h + lq);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int y = 0; y < RB; ++y)
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    acc[y][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[h][c], af[h][y], acc[y][c], 0, 0, 0);
    };
    // whole rounds of the ring, then the rest: a loop with one way out, in which
    // every path to a stage's reads passes the same loads, so that the compiler's
    // own waits stay exact
    int kb = 0;
    for (; kb + S <= KB; kb += S) {
#pragma unroll
        for (int j = 0; j < S; ++j) step(buf[j], buf[(j + S - 1) % S], kb + j);
    }
    if (kb < KB) {
        step(buf[0], buf[3], kb);
        if (kb + 1 < KB) {
            step(buf[1], buf[0], kb + 1);
            if (kb + 2 < KB) step(buf[2], buf[1], kb + 2);
        }
    }
    GFG_WAITCNT(0, 15);                            // the last loads land before the workgroup ends

    // acc[y][c] of lane (l16, lq): row 16 y + l16, columns 16 c + 4 lq .. +3
    OutT* const d = static_cast<OutT*>(p.d);
#pragma unroll
    for (int y = 0; y < RB; ++y) {
        const int r = wm + 16 * y + l16;
        bool ok = r < lim;
        if (LAYOUT == CONTIG) ok = ok && p.meta[row0 + min(r, lim - 1)] == g;
        if (!ok) continue;
        const float sa = p.a_scale[arow + r];
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            const int n = n0 + wn + 16 * c + 4 * lq;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int nn = min(n + i, p.N - 1);
                // adding -0 changes nothing, not even a zero's sign
                v[i] = fmaf(float(acc[y][c][i]) * sa, p.b_scale[int64_t(g) * p.N + nn],
                            LAYOUT == DENSE && p.bias ? p.bias[nn] : -0.0f);
            }
            store4(d + (arow + r) * p.N, n, p.N, v);
        }
    }
}

// The tiles of a workgroup: one, or, under a grid limit, every gridDim.x-th.
template <typename Tile>
__device__ __forceinline__ void walk(unsigned tiles, Tile tile) {
    for (unsigned w = blockIdx.x;;) {
        tile(w);
        w += gridDim.x;
        if (w >= tiles) return;
        __syncthreads();                           // every wave is done with the tile's LDS
    }
}

template <int LAYOUT, int TM, int TN, int S, int WM, int WN, typename OutT>
__global__ __launch_bounds__(WM * WN * 64) void int8_gemm_kernel(I8Params p) {
    walk(p.tiles, [&](unsigned w) { ring_tile<LAYOUT, TM, TN, S, WM, WN, OutT>(p, w); });
}

// ------------------------------------------------------------------ streamed product
//
// 16 RB x 16 CB output tiles whose NW waves split K: wave w takes the 128-byte
// units w, w + NW, ... of the tile's rows through its own ring of D LDS stages,
// filled by direct-to-LDS loads.  No barrier stands between a load and its
// MFMAs, every byte of the tile's rows enters the CU once and leaves the LDS
// once; the waves' sums meet in LDS at the end (integers: exact in any order).
// (Loading the fragments straight into registers instead is slower: a
// fragment's adjacent lanes are adjacent rows, so four lanes touch four cache
// lines: 1 x 7168 x 2304 took twice as long.)  Bound by the launch and the way of
// the first loads, then by a wave's chain of units: 1 x 7168 x 2304 5.9 us with cold
// weights (16.5 MB), 3.5 with warm ones; 128 x 4096 x 4096 9.1.
template <int LAYOUT, int RB, int CB, int NW, int D, typename OutT>
__device__ __forceinline__ void stream_tile(const I8Params& p, unsigned w) {
    constexpr int TM = 16 * RB, TN = 16 * CB;
    constexpr int UNIT = (TM + TN) * TK;           // bytes of a stage: A's rows, then B's
    constexpr int PER = UNIT / 1024;               // loads per stage
    static_assert((D == 2 || D == 4) && PER * D < 64, "ring depth");
    // an array for each stage: the compiler then knows that reading one need
    // not wait for the loads into another
    __shared__ __attribute__((aligned(1024))) uint8_t s0[NW * UNIT], s1[NW * UNIT];
    __shared__ __attribute__((aligned(1024))) uint8_t s2[D > 2 ? NW * UNIT : 1024], s3[D > 2 ? NW * UNIT : 1024];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    GFG_LDS uint8_t* const ring[4] = {(GFG_LDS uint8_t*)s0 + wave * UNIT, (GFG_LDS uint8_t*)s1 + wave * UNIT,
                                      (GFG_LDS uint8_t*)s2 + (D > 2 ? wave * UNIT : 0), (GFG_LDS uint8_t*)s3 + (D > 2 ? wave * UNIT : 0)};
    const unsigned nx = unsigned(p.num_xcd), x = w % nx, per = p.tiles / nx, rem = p.tiles % nx;
    const unsigned item = x * per + min(x, rem) + w / nx;
    const int mt = int(item % unsigned(p.m_tiles)), n0 = int(item / unsigned(p.m_tiles)) * TN;
    int g = 0, row0, lim;
    int64_t region = 0;
    if (LAYOUT == MASKED) {
        g = mt / p.tiles_per_group;
        row0 = (mt - g * p.tiles_per_group) * TM;
        int mm = p.meta[g];
        mm = mm < 0 ? 0 : (mm > p.rows ? int(p.rows) : mm);
        lim = min(TM, mm - row0);
        region = int64_t(g) * p.rows;
    } else {
        row0 = mt * TM;
        lim = int(p.rows - row0 < TM ? p.rows - row0 : TM);
        if (LAYOUT == CONTIG) {
            g = p.meta[row0 & ~127];               // the expert of the aligned 128 rows
            if (g < 0 || g >= p.G) return;
        }
    }
    if (lim <= 0) return;
    g = __builtin_amdgcn_readfirstlane(g);
    lim = __builtin_amdgcn_readfirstlane(lim);
    const int64_t arow = region + row0;
    const int ncols = min(TN, p.N - n0);
    const auto ra = make_rsrc(p.a + arow * p.K, uint32_t(lim) * uint32_t(p.K));
    const auto rb = make_rsrc(p.b + (int64_t(g) * p.N + n0) * p.K, uint32_t(ncols) * uint32_t(p.K));

    // load j: LDS rows 8 j .. +7 of the stage; lane i writes physical chunk
    // i & 7 of row i >> 3 of them, the logical chunk (i & 7) ^ (i >> 3)
    const int kc = ((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t src0 = uint32_t(lane >> 3) * uint32_t(p.K) + uint32_t(kc);
    auto load = [&](GFG_LDS uint8_t* dst, int k) {
        const uint32_t base = k + kc < p.K ? src0 + uint32_t(k) : kOutside;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(j < TM / 8 ? ra : rb, (GFG_LDS void*)(dst + j * 1024), 16,
                                                     base + uint32_t(8 * (j < TM / 8 ? j : j - TM / 8)) * uint32_t(p.K), 0, 0, 0);
    };
    v4i acc[RB][CB] = {};
    auto frag = [&](GFG_LDS uint8_t* src, int row, int chunk) {
        return *reinterpret_cast<GFG_LDS v4i*>(src + (row + l16) * TK + ((chunk ^ (l16 & 7)) << 4));
    };
    // consume a unit, then load the one that takes its place, D units ahead
    auto step = [&](GFG_LDS uint8_t* cur, int k) {
        __builtin_amdgcn_sched_barrier(0);
        GFG_WAITCNT((D - 1) * PER, 15);
        v4i af[2][RB], bf[2][CB];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int f = 0; f < RB; ++f) af[h][f] = frag(cur, 16 * f, 4 * h + lq);
#pragma unroll
            for (int f = 0; f < CB; ++f) bf[h][f] = frag(cur + TM * TK, 16 * f, 4 * h + lq);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int y = 0; y < RB; ++y)
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    acc[y][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[h][c], af[h][y], acc[y][c], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        load(cur, k + D * NW * TK);                // past K: zeros
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int STEP = NW * TK;
#pragma unroll
    for (int d = 0; d < D; ++d) load(ring[d], wave * TK + d * STEP);
    int k = wave * TK;                         // (rounds as above)
    for (; k + (D - 1) * STEP < p.K; k += D * STEP) {
#pragma unroll
        for (int d = 0; d < D; ++d) step(ring[d], k + d * STEP);
    }
    if (k < p.K) {
        step(ring[0], k);
        if constexpr (D > 2) {
            if (k + STEP < p.K) {
                step(ring[1], k + STEP);
                if (k + 2 * STEP < p.K) step(ring[2], k + 2 * STEP);
            }
        }
    }
    GFG_WAITCNT(0, 15);                            // the last loads land before the workgroup ends
    // a wave's sums go where its first stage was
    static_assert(RB * CB * 1024 <= UNIT, "the sums fit a stage");
    auto sums = [&](int w, int i) -> GFG_LDS v4i& { return reinterpret_cast<GFG_LDS v4i*>((GFG_LDS uint8_t*)s0 + w * UNIT)[i * 64 + lane]; };
#pragma unroll
    for (int y = 0; y < RB; ++y)
#pragma unroll
        for (int c = 0; c < CB; ++c) sums(wave, y * CB + c) = acc[y][c];
    __syncthreads();
    OutT* const d = static_cast<OutT*>(p.d);
#pragma unroll
    for (int i0 = 0; i0 < RB * CB; i0 += NW) {
        const int i = i0 + wave;
        if (i >= RB * CB) break;
        v4i v4 = sums(0, i);
#pragma unroll
        for (int w = 1; w < NW; ++w) v4 += sums(w, i);
        const int r = 16 * (i / CB) + l16, n = n0 + 16 * (i % CB) + 4 * lq;
        bool ok = r < lim;
        if (LAYOUT == CONTIG) ok = ok && p.meta[row0 + min(r, lim - 1)] == g;
        if (!ok) continue;
        const float sa = p.a_scale[arow + r];
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int nn = min(n + q, p.N - 1);
            v[q] = fmaf(float(v4[q]) * sa, p.b_scale[int64_t(g) * p.N + nn], LAYOUT == DENSE && p.bias ? p.bias[nn] : -0.0f);
        }
        store4(d + (arow + r) * p.N, n, p.N, v);
    }
}

template <int LAYOUT, int RB, int CB, int NW, int D, typename OutT>
__global__ __launch_bounds__(NW * 64) void int8_stream_kernel(I8Params p) {
    walk(p.tiles, [&](unsigned w) { stream_tile<LAYOUT, RB, CB, NW, D, OutT>(p, w); });
}

// Workgroups of a launch over p.tiles tiles: one for each, or as many as the
// grid limit allows, which is rounded up to whole slots on every XCD.
unsigned workgroups(const I8Params& p) {
    const int lim = grid_limit();
    const unsigned nx = unsigned(p.num_xcd), most = lim > 0 ? (unsigned(lim) + nx - 1) / nx * nx : p.tiles;
    return p.tiles < most ? p.tiles : most;
}

template <int LAYOUT, int RB, int CB, int NW, int D>
int launch_stream(I8Params p, int out_dtype, hipStream_t s) {
    const int groups = LAYOUT == MASKED ? p.G : 1;
    p.tiles_per_group = int((p.rows + 16 * RB - 1) / (16 * RB));
    p.m_tiles = p.tiles_per_group * groups;
    const int64_t tiles = int64_t(p.m_tiles) * ((p.N + 16 * CB - 1) / (16 * CB));
    if (tiles * (NW * 64) >= int64_t(1) << 32) return fail(GFG_EUNSUPPORTED, "the output has too many tiles for one launch");
    p.tiles = unsigned(tiles);
    const dim3 grid(workgroups(p)), block(NW * 64);
    if (out_dtype == GFG_OUT_BF16)
        hipLaunchKernelGGL((int8_stream_kernel<LAYOUT, RB, CB, NW, D, __bf16>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((int8_stream_kernel<LAYOUT, RB, CB, NW, D, _Float16>), grid, block, 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

template <int LAYOUT, int TM, int TN, int S, int WM, int WN>
int launch_ring(I8Params p, int out_dtype, hipStream_t s) {
    const int groups = LAYOUT == MASKED ? p.G : 1;
    p.tiles_per_group = int((p.rows + TM - 1) / TM);
    p.m_tiles = p.tiles_per_group * groups;
    const int64_t tiles = int64_t(p.m_tiles) * ((p.N + TN - 1) / TN);
    if (tiles * (WM * WN * 64) >= int64_t(1) << 32) return fail(GFG_EUNSUPPORTED, "the output has too many tiles for one launch");
    p.tiles = unsigned(tiles);
    const dim3 grid(workgroups(p)), block(WM * WN * 64);
    if (out_dtype == GFG_OUT_BF16)
        hipLaunchKernelGGL((int8_gemm_kernel<LAYOUT, TM, TN, S, WM, WN, __bf16>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((int8_gemm_kernel<LAYOUT, TM, TN, S, WM, WN, _Float16>), grid, block, 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

// ------------------------------------------------------------------ a few tokens, quantized on the way
//
// At most kFewTokens rows of x in 16 or 32 bits: every workgroup quantizes them
// itself, into LDS, while its first weights are on the way (the codes and
// scales are those of the token quantizer, bit for bit), then streams its 32
// weight rows like the kernel above.  One launch instead of two: 7168 x 2304 with
// cold weights (16.5 MB), bf16: 1 token 6.5 us, 9.5 in two launches; 2: 7.0, 9.7; 4:
// 8.0, 9.9 (f32 6.7, 9.0 and 8.1, 9.2).  Every workgroup encodes all rows, half a
// microsecond each, and 5 tokens take 10.0 in two launches, so a few more of them
// would gain nothing.
constexpr int kFewTokens = 4;
constexpr int kFewCodes = 32 * 1024;           // bytes of LDS for the codes

template <int MT, typename X, typename OutT>
__global__ __launch_bounds__(256) void int8_few_kernel(const X* __restrict__ xs, I8Params p) {
    constexpr int NW = 4, D = 4, TN = 32, UNIT = TN * TK, PER = UNIT / 1024;
    __shared__ __attribute__((aligned(1024))) uint8_t s0[NW * UNIT], s1[NW * UNIT], s2[NW * UNIT], s3[NW * UNIT];
    __shared__ __attribute__((aligned(1024))) uint8_t codes[kFewCodes];   // [M][K rounded up to 128], chunks swizzled like a stage's
    __shared__ uint32_t amax[MT][NW];
    __shared__ v4i sums[NW][2][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, lq = lane >> 4;
    GFG_LDS uint8_t* const ring[D] = {(GFG_LDS uint8_t*)s0 + wave * UNIT, (GFG_LDS uint8_t*)s1 + wave * UNIT,
                                      (GFG_LDS uint8_t*)s2 + wave * UNIT, (GFG_LDS uint8_t*)s3 + wave * UNIT};
    const int M = int(p.rows), n0 = int(blockIdx.x) * TN, ncols = min(TN, p.N - n0);
    const auto rb = make_rsrc(p.b + int64_t(n0) * p.K, uint32_t(ncols) * uint32_t(p.K));
    const int kc = ((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t src0 = uint32_t(lane >> 3) * uint32_t(p.K) + uint32_t(kc);
    auto load = [&](GFG_LDS uint8_t* dst, int k) {
        const uint32_t base = k + kc < p.K ? src0 + uint32_t(k) : kOutside;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (GFG_LDS void*)(dst + j * 1024), 16, base + uint32_t(8 * j) * uint32_t(p.K), 0, 0, 0);
    };
    const int chunks = p.K / 8, KP = (p.K + TK - 1) / TK * TK;
    // the rows stay in registers between the maximum and the encoding; they are
    // loaded before the weights, so that they are not waited for behind those
    constexpr int HELD = kFewCodes / 8 / 256 / MT, STEP = NW * TK;
    Chunk<X> held[MT][HELD];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const auto rx = make_rsrc(xs + int64_t(min(m, M - 1)) * p.K, uint32_t(p.K) * uint32_t(sizeof(X)));
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            held[m][i] = Chunk<X>{};
            if (256 * i < chunks) held[m][i].load(rx, (threadIdx.x + 256 * i) * uint32_t(8 * sizeof(X)));   // past K: zeros
        }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < D; ++d) load(ring[d], wave * TK + d * STEP);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t most[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        uint32_t ab = 0;
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (256 * i < chunks) ab = max(ab, chunk_amax(held[m][i]));
        most[m] = wave_reduce(ab, [](uint32_t a, uint32_t b) { return max(a, b); });
    }
    if (lane == 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m) amax[m][wave] = most[m];
    }
    lds_barrier();                             // (the weights stay in flight)
    float scale = 0.0f;                        // of row l16
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (MT > 1 && m >= M) break;
        float s, r;
        row_scale(max(max(amax[m][0], amax[m][1]), max(amax[m][2], amax[m][3])), &s, &r);
        if (l16 == m) scale = s;
        auto put = [&](int c, const Chunk<X>& t) {     // past K the chunk is zeros; a row without a scale is
            const int k = c * 8, chunk = (k >> 4) & 7;
            *reinterpret_cast<u32x2*>(codes + m * KP + (k & ~127) + ((chunk ^ (m & 7)) << 4) + (k & 15)) =
                r == 0.0f ? u32x2{0u, 0u} : chunk_encode(t, r);
        };
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (int(threadIdx.x) + 256 * i < KP / 8) put(int(threadIdx.x) + 256 * i, held[m][i]);
    }
    lds_barrier();

    v4i acc[2] = {};
    const int row = min(l16, M - 1);           // columns past M repeat the last row and are not stored
    auto frag = [&](GFG_LDS uint8_t* src, int rw, int chunk) {
        return *reinterpret_cast<GFG_LDS v4i*>(src + (rw + l16) * TK + ((chunk ^ (l16 & 7)) << 4));
    };
    auto step = [&](GFG_LDS uint8_t* cur, int k) {
        __builtin_amdgcn_sched_barrier(0);
        GFG_WAITCNT((D - 1) * PER, 15);
        v4i af[2], bf[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            af[h] = *reinterpret_cast<GFG_LDS v4i*>((GFG_LDS uint8_t*)codes + row * KP + k + (((4 * h + lq) ^ (row & 7)) << 4));
#pragma unroll
            for (int f = 0; f < 2; ++f) bf[h][f] = frag(cur, 16 * f, 4 * h + lq);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[h][c], af[h], acc[c], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        load(cur, k + D * STEP);               // past K: zeros
        __builtin_amdgcn_sched_barrier(0);
    };
    int k = wave * TK;                         // (rounds as above)
    for (; k + (D - 1) * STEP < p.K; k += D * STEP) {
#pragma unroll
        for (int d = 0; d < D; ++d) step(ring[d], k + d * STEP);
    }
    if (k < p.K) {
        step(ring[0], k);
        if (k + STEP < p.K) {
            step(ring[1], k + STEP);
            if (k + 2 * STEP < p.K) step(ring[2], k + 2 * STEP);
        }
    }
    GFG_WAITCNT(0, 15);                        // the last loads land before the workgroup ends
    sums[wave][0][lane] = acc[0];
    sums[wave][1][lane] = acc[1];
    __syncthreads();
    if (wave >= 2 || l16 >= M) return;
    const v4i total = sums[0][wave][lane] + sums[1][wave][lane] + sums[2][wave][lane] + sums[3][wave][lane];
    const int n = n0 + 16 * wave + 4 * lq;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int nn = min(n + i, p.N - 1);
        v[i] = fmaf(float(total[i]) * scale, p.b_scale[nn], p.bias ? p.bias[nn] : -0.0f);
    }
    store4(static_cast<OutT*>(p.d) + int64_t(l16) * p.N, n, p.N, v);
}

template <int MT, typename X>
void launch_few_rows(const void* x, const I8Params& p, int out_dtype, hipStream_t s) {
    const dim3 grid(p.tiles), block(256);
    if (out_dtype == GFG_OUT_BF16)
        hipLaunchKernelGGL((int8_few_kernel<MT, X, __bf16>), grid, block, 0, s, static_cast<const X*>(x), p);
    else
        hipLaunchKernelGGL((int8_few_kernel<MT, X, _Float16>), grid, block, 0, s, static_cast<const X*>(x), p);
}

// Whether M rows of K codes go this way: a workgroup has one tile, so not under
// a grid limit that is below their number (walking tiles in this kernel costs
// it 0.5 us where there is no limit).
bool few(I8Params* p) {
    p->tiles = unsigned((p->N + 31) / 32);
    const int64_t rows = p->rows == 3 ? 4 : p->rows;       // (three run as four)
    return rows <= kFewTokens && rows * ((p->K + TK - 1) / TK * TK) <= kFewCodes && workgroups(*p) == p->tiles;
}

template <typename X>
int launch_few(const void* x, const I8Params& p, int out_dtype, hipStream_t s) {
    if (p.rows == 1) launch_few_rows<1, X>(x, p, out_dtype, s);
    else if (p.rows == 2) launch_few_rows<2, X>(x, p, out_dtype, s);
    else launch_few_rows<kFewTokens, X>(x, p, out_dtype, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

// The launches with too few 256 x 256 tiles, by how many tiles of each size
// there are (M x N x K, us, the chosen tile first):
//  * up to 16 rows: the streamed 16 x 32 tile (cold weights, 32 x 32 second: 1 x
//    1024 x 7168: 5.6, 6.5; 4 x 2048 x 16384: 14.9, 16.1; 1 x 4096 x 4096: 6.6, 7.1; 1 x
//    7168 x 2304: 5.9, 5.9; but 1 x 28672 x 4096, 896 tiles: 28.7, 25.3), or 32 x 32 up to
//    32 rows (32 x 4096 x 4096: 5.9, 64 x 64 9.4);
//  * 192 tiles of 128 x 128 or more: those (512 x 7168 x 2304, 224 of them: 16.0,
//    64 x 64 20.0; 1024 x 4096 x 4096, 256: 23.5, 30.8);
//  * up to 512 tiles of 32 x 32: those, streamed (128 x 4096 x 4096: 9.1, 64 x 64
//    10.0; 300 x 770 x 4096: 5.9, 9.8; 4096 x 64 x 16384: 22.4, 37.6);
//  * else 64 x 64 (2000 x 300 x 16384: 28.4, 32 x 32 50.4; 128 x 7168 x 2304: 7.6,
//    11.2; 512 x 4096 x 4096: 17.5, 29.2, 128 x 128 21.0).
template <int LAYOUT>
int launch_small(const I8Params& p, int out_dtype, hipStream_t s) {
    auto tiles = [&](int64_t tm, int64_t tn) {
        return (p.rows + tm - 1) / tm * (LAYOUT == MASKED ? p.G : 1) * ((p.N + tn - 1) / tn);
    };
    if (p.rows <= 16) return launch_stream<LAYOUT, 1, 2, 4, 4>(p, out_dtype, s);
    if (p.rows <= 32) return launch_stream<LAYOUT, 2, 2, 4, 2>(p, out_dtype, s);
    if (tiles(128, 128) >= 192) return launch_ring<LAYOUT, 128, 128, 4, 2, 4>(p, out_dtype, s);
    if (tiles(32, 32) <= 512) return launch_stream<LAYOUT, 2, 2, 4, 2>(p, out_dtype, s);
    return launch_ring<LAYOUT, 64, 64, 4, 2, 2>(p, out_dtype, s);
}

// Launch the product on the tile that suits it: the 256 x 256 kernel (whose
// tiles have 192 rows where that fills the CUs better) wherever tiles of
// 128 x 128 would need a second round over the CUs.  Measured, us, the 256
// kernel and the smaller tiles' own choice: 2000 x 4096 x 4096 (512 tiles of
// 128 x 128) 41.5, 48.4; 768 x 7168 x 2304 (336) 26.4, 27.9; 700 x 6144 x 4096 (288) 38.4,
// 40.0; 2048 x 2104 x 1024 (272) 17.1, 17.9; but 1024 x 4096 x 4096 (256) 38.3, 23.5;
// 1920 x 2048 x 7168 (240) 61.8, 37.1.  Just past the threshold tiles of 64 x 64 would
// be faster than both (34.5 and 15.4 at 288 and 272).  The masked layout is counted
// by its capacity, since the live rows are device data: with 1 to 32 of 1024 rows in
// each of 8 groups, N = 2048, K = 7168, the 256 kernel takes 69 us where the smaller
// tiles take 59 to 63; with 128 rows 74 and 85, with 1024 104 and 171.
// `p` holds everything but the tile counts.
int launch_i8(const char* fn, I8Params p, int layout, int out_dtype, hipStream_t s) {
    const int groups = layout == MASKED ? p.G : 1;
    const int64_t t128 = (p.rows + 127) / 128 * groups, n128 = (int64_t(p.N) + 127) / 128;
    const bool fits = p.N <= 1 << 22;
    const int choice = tile_shape_choice();
    if (choice == GFG_TILE_256x256 && !fits)
        return fail(GFG_EUNSUPPORTED, "%s: the 256 x 256 tile needs N=%d at most 2^22", fn, p.N);
    int cus = 0;
    if (int rc = device_cus(&cus)) return rc;
    if (choice == GFG_TILE_256x256 || (choice == GFG_TILE_AUTO && fits && t128 * n128 > cus)) {
        p.m_tiles = int(t128);                 // (read for the contiguous layout: the 128-row candidates)
        return launch_int8_256(p, layout, out_dtype, s);
    }
    if (layout == DENSE) return launch_small<DENSE>(p, out_dtype, s);
    if (layout == CONTIG) return launch_small<CONTIG>(p, out_dtype, s);
    return launch_small<MASKED>(p, out_dtype, s);
}

I8Params product(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale, const float* bias,
                 const int32_t* meta, void* d, int64_t rows, int64_t N, int64_t K, int G) {
    I8Params p{};
    p.a = reinterpret_cast<const uint8_t*>(a);
    p.a_scale = a_scale;
    p.b = reinterpret_cast<const uint8_t*>(b);
    p.b_scale = b_scale;
    p.bias = bias;
    p.meta = meta;
    p.d = d;
    p.rows = rows;
    p.N = int(N);
    p.K = int(K);
    p.G = G;
    p.group_m = locality_group_m();
    p.num_xcd = locality_num_xcd();
    return p;
}

// ------------------------------------------------------------------ argument checks
constexpr int64_t kMaxK = (int64_t(1) << 17) - 16;     // |sum| <= 2^14 K stays below 2^31
constexpr int64_t kMaxN = int64_t(1) << 28;
constexpr int64_t kMaxRowTiles = 65535;                // of 128 rows

int check_quant(const char* fn, const void* x, int32_t in_dtype, int64_t M, int64_t K, const void* q, const void* scale) {
    if (in_dtype != GFG_IN_F32 && in_dtype != GFG_IN_BF16 && in_dtype != GFG_IN_F16)
        return fail(GFG_EINVAL, "%s: in_dtype %d is not a GFG_IN_* value", fn, in_dtype);
    if (M < 0 || K <= 0) return fail(GFG_EINVAL, "%s: bad sizes M=%lld K=%lld", fn, (long long)M, (long long)K);
    if (K % 16 || K > kMaxK)
        return fail(GFG_EUNSUPPORTED, "%s: K=%lld must be a multiple of 16 and at most %lld", fn, (long long)K,
                    (long long)kMaxK);
    if (M >= int64_t(1) << 31) return fail(GFG_EUNSUPPORTED, "%s: M=%lld is 2^31 or more", fn, (long long)M);
    if (M == 0) return GFG_OK;
    if (!x || !q || !scale) return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(q)) % 16 || reinterpret_cast<uintptr_t>(scale) % 4)
        return fail(GFG_EINVAL, "%s: x and q must be 16-byte aligned, scale 4-byte aligned", fn);
    return GFG_OK;
}

// Sizes of a product; *empty is set when there is nothing to compute.
int check_product(const char* fn, int64_t rows, int64_t N, int64_t K, int64_t G, int32_t out_dtype, bool* empty) {
    *empty = false;
    if (out_dtype != GFG_OUT_BF16 && out_dtype != GFG_OUT_F16)
        return fail(GFG_EINVAL, "%s: out_dtype %d is not GFG_OUT_BF16 or GFG_OUT_F16", fn, out_dtype);
    if (rows < 0 || N <= 0 || K <= 0 || G <= 0 || G > 65535)
        return fail(GFG_EINVAL, "%s: bad sizes rows=%lld N=%lld K=%lld G=%lld", fn, (long long)rows, (long long)N,
                    (long long)K, (long long)G);
    if (K % 16 || K > kMaxK)
        return fail(GFG_EUNSUPPORTED, "%s: K=%lld must be a multiple of 16 and at most %lld", fn, (long long)K,
                    (long long)kMaxK);
    if (N > kMaxN) return fail(GFG_EUNSUPPORTED, "%s: N=%lld above 2^28", fn, (long long)N);
    if (rows > kMaxRowTiles * 128)
        return fail(GFG_EUNSUPPORTED, "%s: %lld rows, at most %lld", fn, (long long)rows, (long long)(kMaxRowTiles * 128));
    *empty = rows == 0;
    return GFG_OK;
}

int check_operands(const char* fn, const void* a, const void* a_scale, const void* b, const void* b_scale,
                   const void* meta, bool need_meta, const void* d) {
    if (!a || !a_scale || !b || !b_scale || !d || (need_meta && !meta))
        return fail(GFG_EINVAL, "%s: null pointer argument", fn);
    if ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) % 16)
        return fail(GFG_EINVAL, "%s: a and b must be 16-byte aligned", fn);
    if ((reinterpret_cast<uintptr_t>(a_scale) | reinterpret_cast<uintptr_t>(b_scale) | reinterpret_cast<uintptr_t>(meta)) % 4 ||
        reinterpret_cast<uintptr_t>(d) % 8)
        return fail(GFG_EINVAL, "%s: scales and metadata must be 4-byte aligned, d 8-byte aligned", fn);
    return GFG_OK;
}

int quantize(const void* x, int32_t in_dtype, int64_t M, int64_t K, uint8_t* q, float* scale, hipStream_t s) {
    if (in_dtype == GFG_IN_F32) launch_quant<float>(x, q, scale, M, int(K), s);
    else if (in_dtype == GFG_IN_BF16) launch_quant<__bf16>(x, q, scale, M, int(K), s);
    else launch_quant<_Float16>(x, q, scale, M, int(K), s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(GFG_EHIP, "kernel launch failed: %s", hipGetErrorString(e));
    return GFG_OK;
}

}  // namespace
}  // namespace gfg

using namespace gfg;

extern "C" int int8_quantize_token_device(const void* x, int32_t in_dtype, int64_t M, int64_t K, int8_t* q,
                                          float* scale, void* stream) {
    clear_error();
    if (int rc = check_quant("int8_quantize_token_device", x, in_dtype, M, K, q, scale)) return rc;
    if (M == 0) return GFG_OK;
    return quantize(x, in_dtype, M, K, reinterpret_cast<uint8_t*>(q), scale, static_cast<hipStream_t>(stream));
}

extern "C" int int8_gemm(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
                         const float* bias, void* d, int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* stream) {
    clear_error();
    const char* fn = "int8_gemm";
    bool empty;
    if (int rc = check_product(fn, M, N, K, 1, out_dtype, &empty)) return rc;
    if (empty) return GFG_OK;
    if (int rc = check_operands(fn, a, a_scale, b, b_scale, bias, false, d)) return rc;
    return launch_i8(fn, product(a, a_scale, b, b_scale, bias, nullptr, d, M, N, K, 1), DENSE, out_dtype,
                     static_cast<hipStream_t>(stream));
}

extern "C" int64_t int8_linear_workspace_bytes(int64_t M, int64_t K) {
    return M > 0 && K > 0 ? M * ((K + 15) / 16 * 16) + M * 4 : 0;
}

extern "C" int int8_linear(const void* x, int32_t in_dtype, const int8_t* b, const float* b_scale, const float* bias,
                           void* d, int64_t M, int64_t N, int64_t K, int32_t out_dtype, void* workspace,
                           int64_t workspace_bytes, void* stream) {
    clear_error();
    const char* fn = "int8_linear";
    bool empty;
    if (int rc = check_product(fn, M, N, K, 1, out_dtype, &empty)) return rc;
    if (in_dtype != GFG_IN_F32 && in_dtype != GFG_IN_BF16 && in_dtype != GFG_IN_F16)
        return fail(GFG_EINVAL, "%s: in_dtype %d is not a GFG_IN_* value", fn, in_dtype);
    if (empty) return GFG_OK;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16)
        return fail(GFG_EINVAL, "%s: workspace must be a 16-byte aligned device pointer", fn);
    if (workspace_bytes < int8_linear_workspace_bytes(M, K))
        return fail(GFG_EINVAL, "%s: workspace of %lld bytes, %lld are needed", fn, (long long)workspace_bytes,
                    (long long)int8_linear_workspace_bytes(M, K));
    uint8_t* const q = static_cast<uint8_t*>(workspace);
    float* const scale = reinterpret_cast<float*>(q + M * K);
    if (int rc = check_quant(fn, x, in_dtype, M, K, q, scale)) return rc;
    if (int rc = check_operands(fn, q, scale, b, b_scale, bias, false, d)) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (I8Params p = product(nullptr, nullptr, b, b_scale, bias, nullptr, d, M, N, K, 1); few(&p)) {
        if (in_dtype == GFG_IN_F32) return launch_few<float>(x, p, out_dtype, s);
        if (in_dtype == GFG_IN_BF16) return launch_few<__bf16>(x, p, out_dtype, s);
        return launch_few<_Float16>(x, p, out_dtype, s);
    }
    if (int rc = quantize(x, in_dtype, M, K, q, scale, s)) return rc;
    return launch_i8(fn, product(reinterpret_cast<const int8_t*>(q), scale, b, b_scale, bias, nullptr, d, M, N, K, 1), DENSE,
                     out_dtype, s);
}

extern "C" int grouped_int8_gemm_contiguous(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
                                            const int32_t* grouped_layout, void* d, int64_t M, int64_t N, int64_t K,
                                            int32_t G, int32_t out_dtype, void* stream) {
    clear_error();
    const char* fn = "grouped_int8_gemm_contiguous";
    bool empty;
    if (int rc = check_product(fn, M, N, K, G, out_dtype, &empty)) return rc;
    if (empty) return GFG_OK;
    if (int rc = check_operands(fn, a, a_scale, b, b_scale, grouped_layout, true, d)) return rc;
    const int64_t tiles = (M + 127) / 128;
    if (tiles > 4096) return fail(GFG_EUNSUPPORTED, "%s: M=%lld is more than 4096 tiles of 128 rows", fn, (long long)M);
    return launch_i8(fn, product(a, a_scale, b, b_scale, nullptr, grouped_layout, d, M, N, K, G), CONTIG, out_dtype,
                     static_cast<hipStream_t>(stream));
}

extern "C" int grouped_int8_gemm_masked(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
                                        const int32_t* masked_m, void* d, int32_t G, int64_t M_max, int64_t N, int64_t K,
                                        int32_t out_dtype, void* stream) {
    clear_error();
    const char* fn = "grouped_int8_gemm_masked";
    bool empty;
    if (int rc = check_product(fn, M_max, N, K, G, out_dtype, &empty)) return rc;
    if (empty) return GFG_OK;
    if (int rc = check_operands(fn, a, a_scale, b, b_scale, masked_m, true, d)) return rc;
    const int64_t tiles = (M_max + 127) / 128;
    if (tiles > 4096 || tiles * G > 4096)
        return fail(GFG_EUNSUPPORTED, "%s: G=%d x M_max=%lld is more than 4096 tiles of 128 rows", fn, G, (long long)M_max);
    return launch_i8(fn, product(a, a_scale, b, b_scale, nullptr, masked_m, d, M_max, N, K, G), MASKED, out_dtype,
                     static_cast<hipStream_t>(stream));
}
